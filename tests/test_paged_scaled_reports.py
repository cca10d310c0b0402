"""fa_kv_append_scaled: which sequences it reports."""
import pytest
import torch

from tests.test_paged import fa  # noqa: F401  (the fixture)
from tests.test_paged_scaled import Batch8

gpu = pytest.mark.gpu


def detail(fa):  # noqa: F811
    with pytest.raises(fa.FAError) as e:
        fa.default_workspace("cuda").check()
    assert e.value.status == fa.ERR_DEVICE_CHECK
    return str(e.value)


@gpu
@pytest.mark.parametrize("B,bad", [(3, 2), (256, 255), (257, 256), (300, 299), (700, 300), (700, 600), (2048, 1500)])
@pytest.mark.parametrize("rows", ["all", "bad alone"])
@pytest.mark.parametrize("queries", [False, True])
def test_a_bad_sequence_is_reported_wherever_it_stands(fa, B, bad, rows, queries):  # noqa: F811
    """More new tokens than kv_len says: reported, with or without queries; the others' tokens are written."""
    new = [1] * B if rows == "all" else [1] + [0] * (B - 1)
    new[bad] = 2
    bt = Batch8(new, [20] * B, 2, 64, 16)
    (kc, vc, table, kv, qs), s = bt.device8()
    kv[bad] = 1
    x = torch.randn(bt.total, 6, 64, device="cuda").to(torch.bfloat16)
    fa.kv_append(x[:, :2] if queries else None, x[:, 2:4], x[:, 4:], kc, vc, table, kv, qs, **s)
    assert f"sequence {bad}" in detail(fa)
    for b in range(B):
        if new[b] and b != bad:
            want = (x[bt.q_start[b], 4:].float().cpu() / s["v_scale"][bt.table[b, 1]].cpu()[:, None]).to(torch.float8_e4m3fn)
            assert torch.equal(vc[bt.table[b, 1], :, 3].cpu().view(torch.uint8), want.view(torch.uint8)), b
