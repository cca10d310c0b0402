"""Calls at the edges of what the paged cache and the sink window take: batches
without a token, the widest masks, rows that are repeated or already in place,
more sequences than attention takes, and numbers past 32 bits."""
import numpy as np
import pytest
import torch

from tests.test_paged import Batch, compare, fa, reference, run  # noqa: F401  (fa: the fixture)

gpu = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(window=2**31), dict(window=2**32 + 5), dict(sinks=2**32 + 1), dict(prefix_len=2**40),
                                dict(window=-2**31 - 1)], ids=str)
def test_block_mask_refuses_more_than_32_bits(fa, kw):  # noqa: F811
    """A field of 32 bits would take the low ones: a window of 5."""
    with pytest.raises(ValueError, match="32-bit"):
        fa.block_mask("sink_window", 1, 1, 8, 8, device="cpu", **kw)


def test_packing_refuses_more_than_32_bits(fa):  # noqa: F811
    for values in ((1, 2**31, 0, 0, 0, 0, 0), (1, -2**31 - 1, 0, 0, 0, 0, 0)):
        with pytest.raises(ValueError, match="32 bits"):
            fa._packed(fa._MASK, "the mask", *values)


@gpu
def test_paged_refuses_more_than_32_bits(fa):  # noqa: F811
    bt = Batch([1, 1], [20, 30], 2, 64, 16)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    for kw in (dict(mask="sliding_window", window=2**31), dict(mask="sink_window", sinks=2**32 + 1), dict(max_q_len=2**31),
               dict(shared_len=2**31), dict(score="rel_bias", rel_max=2**31)):
        with pytest.raises(ValueError):
            fa.fwd_paged(q, *bt.device(), **kw)
    with pytest.raises(fa.FAError, match="finite"):            # infinite in 32 bits
        fa.fwd_paged(q, *bt.device(), score="softcap", softcap=1e300)


@gpu
@pytest.mark.parametrize("shared", [0, 64])
@pytest.mark.parametrize("max_q", [1, 40])
def test_no_sequence_has_a_token(fa, max_q, shared):  # noqa: F811
    """Rows of padding only: nothing is written, nothing is reported."""
    bt = Batch([0, 0, 0], [shared + 5, 0, 300], 2, 64, 16, shared=0, pad=6)
    dev = bt.device()
    q = torch.full((6, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 3), torch.full((6, 4), 3.0, device="cuda")
    fa.fwd_paged(q, *dev, max_q_len=max_q, shared_len=shared, out=out, lse=lse)
    assert (out == 3).all() and (lse == 3).all()
    k0 = [x.clone() for x in dev[:2]]
    fa.kv_append(q, q[:, :2], q[:, 2:], *dev, q_out=out)
    assert (out == 3).all() and all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(k0, dev))
    fa.default_workspace("cuda").check()


@gpu
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("shared", [0, 80])
@pytest.mark.parametrize("mask,window,sinks", [("sliding_window", 2**31 - 1, 0), ("sink_window", 2**31 - 1, 2**31 - 1),
                                               ("sink_window", 0, 2**31 - 1), ("sink_window", 2**31 - 300, 3)])
def test_widest_masks(fa, n, shared, mask, window, sinks):  # noqa: F811
    run(fa, Batch([n, n, 1], [shared + n + 300, shared + n, shared + 600], 2, 64, 16, shared=shared), 6, mask, window, sinks)


@gpu
def test_append_repeated_rows_in_place_slices_and_many_sequences(fa):  # noqa: F811
    B = 5000                                       # more than attention takes in one call
    bt = Batch([b % 2 for b in range(B)], [(b * 7) % 40 + 1 for b in range(B)], 2, 64, 16)
    kc, vc, table, kv, qs = bt.device()
    T = bt.total
    fused = torch.randn(T, 6, 64, device="cuda").to(torch.bfloat16)
    one = torch.randn(1, 2, 64, device="cuda").to(torch.bfloat16)
    angle = torch.rand(64, 32, device="cuda") * 6
    kw = dict(cos=angle.cos(), sin=angle.sin())
    q = fused[:, :4]
    want = fa.kv_append(q, fused[:, 4:], one.expand(T, 2, 64), kc, vc, table, kv, qs, **kw)
    keys = fused[:, 4:].clone()
    got = fa.kv_append(q, fused[:, 4:], one.expand(T, 2, 64), kc, vc, table, kv, qs, q_out=q, **kw)
    fa.default_workspace("cuda").check()
    assert got is q and torch.equal(q, want) and torch.equal(fused[:, 4:], keys)
    new = np.flatnonzero(np.array(bt.new))
    at = np.array(bt.kv)[new] - 1
    pages = torch.from_numpy(bt.table[new, at // 16]).long().cuda()
    slots = torch.from_numpy(at % 16).cuda()
    assert torch.equal(vc[pages, :, slots], one.expand(T, 2, 64))
    a, b = keys[..., :32].float(), keys[..., 32:].float()
    c, s = (x[torch.from_numpy(at).cuda()][:, None] for x in (angle.cos(), angle.sin()))
    y, mag = torch.cat([a * c - b * s, a * s + b * c], -1), torch.cat([(a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()], -1)
    # products and one sum in fp32 on both sides, then half a bf16 step
    assert ((kc[pages, :, slots].float() - y).abs() <= 2.0 ** -8 * y.abs() + 6 * 2.0 ** -24 * mag).all()


@gpu
@pytest.mark.parametrize("n", [1, 40])
def test_output_in_place(fa, n):  # noqa: F811
    """out may be q: every row is read before it is written."""
    for shared in (0, 96):
        bt = Batch([n] * 5, [shared + n + 700 * b for b in range(5)], 2, 64, 16, shared=shared)
        dev, q = bt.device(), torch.from_numpy(bt.queries(4)).cuda().to(torch.bfloat16)
        ref = reference(bt, bt.queries(4), "causal", 0, 0)
        _, lse = fa.fwd_paged(q, *dev, max_q_len=n, shared_len=shared, out=q)
        fa.default_workspace("cuda").check()
        compare((q, lse), ref)
