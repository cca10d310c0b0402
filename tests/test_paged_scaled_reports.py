"""fa_kv_append_scaled: which sequences it reports, and what a token without a place leaves alone."""
import numpy as np
import pytest
import torch

from tests.test_paged import fa  # noqa: F401  (the fixture)
from tests.test_paged_scaled import Batch8, least_scale

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


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_a_token_outside_the_tables_counts_nowhere(fa, D):  # noqa: F811
    """Its slot keeps its bytes; scales and the earlier and written codes are those of the tokens that have a place."""
    bt = Batch8([3, 2], [20, 40], 2, D, 16)
    (kc, vc, table, kv, qs), s = bt.device8()
    x = torch.randn(5, 8, D, device="cuda").to(torch.bfloat16)
    x[1] *= 1000                                 # the largest by far, and no power of two away from the others
    ang = torch.rand(50, 32, device="cuda")
    pos = torch.tensor([4, 50, 49, 7, -1], dtype=torch.int32, device="cuda")
    before = [z.view(torch.uint8).cpu().numpy().copy() for z in (kc, vc)]
    fa.kv_append(x[:, :4], x[:, 4:6], x[:, 6:], kc, vc, table, kv, qs, **s, cos=torch.cos(ang), sin=torch.sin(ang),
                 positions=pos)
    detail(fa)
    c, n = ang.cos().double().cpu().numpy(), ang.sin().double().cpu().numpy()
    xs = x.double().cpu().numpy()
    after = [z.view(torch.uint8).cpu().numpy() for z in (kc, vc)]
    untouched = np.ones(kc.shape[0], bool)
    # (sequence, rows written with their slots, slots left alone, earlier tokens) of each page that has new tokens
    for b, page, written, skipped, earlier in ((0, 1, ((0, 1), (2, 3)), (2,), 1), (1, 2, ((3, 6),), (7,), 6)):
        pg = bt.table[b, page]
        untouched[pg] = False
        for h in range(2):
            for e, (name, cols) in enumerate((("k", 4), ("v", 6))):
                rows = []
                for r, _ in written:
                    y = xs[r, cols + h].copy()
                    if name == "k":
                        p, a, z = int(pos[r]), y[:32].copy(), y[32:64].copy()
                        y[:32], y[32:64] = a * c[p] - z * n[p], z * c[p] + a * n[p]
                    rows.append(y)
                codes0, old = getattr(bt, name + "_codes")[pg, h], float(getattr(bt, name + "_scale")[pg, h])
                scale = max(least_scale(np.abs(rows).max()), old)
                assert s[name + "_scale"][pg, h].item() == scale
                got = (kc, vc)[e][pg, h].float().double().cpu().numpy()
                want = torch.from_numpy((codes0[:earlier] * (old / scale)).astype(np.float32)).to(torch.float8_e4m3fn)
                assert np.array_equal(got[:earlier], want.double().numpy())
                for (_, slot), y in zip(written, rows):
                    # half a step of e4m3, and of fp32 3 x 2^-24 of 1300 at most
                    near = 2.0 ** (np.floor(np.log2(np.clip(np.abs(y / scale), 2.0 ** -6, 448))) - 4) + 2.0 ** -12
                    assert (np.abs(got[slot] - y / scale) <= near).all()
                for slot in [*skipped, *range(earlier + 3 - b, 16)]:
                    assert np.array_equal(after[e][pg, h, slot], before[e][pg, h, slot]), (b, name, h, slot)
    for e in range(2):
        assert np.array_equal(after[e][untouched], before[e][untouched])
