"""Attention under a sliding window with sink tokens (mask "sink_window"):
query i sees key j when i >= j and (i - j <= window or j < sinks).

CPU: the oracle's predicate against a dense one and against the masks it
reduces to, its gradient against differences, and the refusals.  GPU: the
BlockMask and its transpose bit for bit, the forward (bf16, fp32, decoding)
and the backward against the oracle.

Tolerances are the forward's and backward's own (tests/parity.py,
tests/test_bwd_gpu.py): the mask changes which products are summed, not how
they are rounded.
"""
import ctypes

import numpy as np
import pytest

import oracle
from block_sparse_attention_fa_gb300 import synth
from tests import parity

gpu = pytest.mark.gpu


def dense(q_len, kv_len, window, sinks):
    i, j = np.arange(q_len)[:, None], np.arange(kv_len)[None]
    return (i >= j) & ((i - j <= window) | (j < sinks))


def reference(q, k, v, see):
    """Plain float64 attention under a dense mask; rows that see nothing give 0 and -inf."""
    g = q.shape[1] // k.shape[1]
    k, v = np.repeat(k, g, 1).astype(np.float64), np.repeat(v, g, 1).astype(np.float64)
    x = np.where(see, q.astype(np.float64) @ k.swapaxes(-1, -2) / np.sqrt(q.shape[-1]), -np.inf)
    m = x.max(-1, keepdims=True)
    p = np.exp(x - np.where(np.isfinite(m), m, 0))
    s = p.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        return p @ v / np.where(s > 0, s, 1), (m + np.log(s))[..., 0]


# --------------------------------------------------------------------- oracle
@pytest.mark.parametrize("q_len,kv_len,window,sinks", [(9, 9, 2, 3), (1, 1, 0, 0), (12, 7, 1, 2), (7, 12, 0, 20),
                                                       (40, 40, 100, 1), (20, 20, 0, 0)])
def test_oracle_against_dense(q_len, kv_len, window, sinks):
    q = synth.standard_normal(3, (1, 2, q_len, 4))
    k, v = synth.standard_normal(4, (1, 1, kv_len, 4)), synth.standard_normal(5, (1, 1, kv_len, 4))
    o, lse = oracle.fwd(q, k, v, mask="sink_window", window=window, prefix_len=sinks)
    ro, rl = reference(q, k, v, dense(q_len, kv_len, window, sinks))
    np.testing.assert_allclose(o, ro, atol=1e-13)
    np.testing.assert_allclose(lse, rl, atol=1e-13)


def test_oracle_reductions():
    q, k, v = (synth.standard_normal(s, (1, 2, 30, 8)) for s in (1, 2, 3))
    sink = lambda w, s: oracle.fwd(q, k, v, mask="sink_window", window=w, prefix_len=s)[0]   # noqa: E731
    assert np.array_equal(sink(4, 0), oracle.fwd(q, k, v, mask="sliding_window", window=4)[0])
    causal = oracle.fwd(q, k, v, mask="causal")[0]
    assert np.array_equal(sink(29, 0), causal) and np.array_equal(sink(0, 30), causal)


def test_oracle_gradient_against_differences():
    """Central differences of sum(O * dO), step h = 1e-5: their error is h^2 times a third derivative plus
    2^-53 / h, below 1e-8 for values of order 1."""
    rng = np.random.default_rng(0)
    q, g = rng.standard_normal((1, 2, 7, 4)), rng.standard_normal((1, 2, 7, 4))
    k, v = rng.standard_normal((1, 1, 7, 4)), rng.standard_normal((1, 1, 7, 4))
    q, k, v, g = (x.astype(np.float32).astype(np.float64) for x in (q, k, v, g))
    see = dense(7, 7, 1, 2)
    grads = oracle.bwd(q, k, v, g, mask="sink_window", window=1, prefix_len=2)
    h = 1e-5
    for which, got in enumerate(grads):
        args = [q, k, v]
        num = np.zeros_like(args[which])
        for at in np.ndindex(num.shape):
            for sign in (1, -1):
                x = [a.copy() for a in args]
                x[which][at] += sign * h
                num[at] += sign * (reference(*x, see)[0] * g).sum() / (2 * h)
        np.testing.assert_allclose(got, num, atol=1e-7)


# ------------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def fa():
    from block_sparse_attention_fa_gb300 import build, fa as fam
    try:
        build.build()
    except RuntimeError as e:  # no CUDA toolkit on this host
        pytest.skip(str(e))
    fam.load_library()
    return fam


@pytest.mark.parametrize("window,sinks,words", [(-1, 0, b"window"), (4, -1, b"sink")])
def test_refusals(fa, window, sinks, words):
    s = fa.BlockMaskStruct()
    s.B = s.H = 1
    s.q_len = s.kv_len = 256
    s.block_q = s.block_kv = 128
    s.nq = s.nkv = 2
    s.kv_num_blocks = s.kv_indices = s.full_kv_num_blocks = s.full_kv_indices = 0x10000
    s.mask.kind, s.mask.window, s.mask.prefix_len = fa.MASK_KINDS["sink_window"], window, sinks
    lib = fa.load_library()
    assert lib.fa_block_mask_build(ctypes.byref(s), ctypes.c_void_p(0x10000), None) == fa.ERR_INVALID_ARG
    assert words in lib.fa_last_error()


def test_binding_refuses_sinks_elsewhere(fa):
    for kw in (dict(mask="causal", sinks=4), dict(mask="sink_window", sinks=4, prefix_len=4)):
        with pytest.raises(ValueError):
            fa.block_mask(B=1, H=1, q_len=8, kv_len=8, device="cpu", **kw)


# ------------------------------------------------------------------------ GPU
SIZES = [(1, 1, 0, 0), (300, 300, 40, 4), (1000, 1000, 128, 130), (129, 129, 0, 1), (700, 700, 2000, 3),
         (513, 513, 127, 0), (640, 640, 255, 128), (260, 900, 10, 300), (900, 260, 100, 5), (257, 257, 1, 2**31 - 1),
         (400, 400, 2**31 - 1, 7)]


@gpu
@pytest.mark.parametrize("q_len,kv_len,window,sinks", SIZES)
def test_block_mask_bits(fa, q_len, kv_len, window, sinks):
    bm = fa.block_mask("sink_window", 1, 1, q_len, kv_len, window=window, sinks=sinks)
    cols = bm.cols()
    fa.default_workspace("cuda").check()
    ref = oracle.block_mask(mask="sink_window", B=1, H=1, q_len=q_len, kv_len=kv_len, window=window, prefix_len=sinks)
    got = bm.numpy()
    for name, x in got.items():
        assert np.array_equal(x, ref[name]), name
    # the transpose lists the same tiles
    for num, idx, knum, kidx in (("q_num_blocks", "q_indices", "kv_num_blocks", "kv_indices"),
                                 ("full_q_num_blocks", "full_q_indices", "full_kv_num_blocks", "full_kv_indices")):
        rows = {(r, int(c)) for r in range(bm.nq) for c in got[kidx][0, 0, r, : got[knum][0, 0, r]]}
        n, x = cols[num].cpu().numpy(), cols[idx].cpu().numpy()
        assert {(int(r), c) for c in range(bm.nkv) for r in x[0, 0, c, : n[0, 0, c]]} == rows
        assert all((x[0, 0, c, n[0, 0, c]:] == -1).all() for c in range(bm.nkv))


def _case(dtype="bf16", B=2, Hq=4, Hkv=2, T=300, D=128, **kw):
    return synth.Workload(name="sinks", dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, T=T, D=D, mask="sink_window", seed=61, **kw)


def _okw(window, sinks):
    return dict(mask="sink_window", window=window, prefix_len=sinks)


SCORES = [("none", {}), ("softcap", {"softcap": 5.0}), ("alibi", {}), ("rel_bias", {"rel_max": 40}),
          ("alibi_softcap", {"softcap": 4.0})]


@gpu
@pytest.mark.parametrize("q_len,kv_len,window,sinks", SIZES)
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("fp32", 64), ("fp32", 128)])
def test_forward_sizes(fa, dtype, D, q_len, kv_len, window, sinks):
    w = _case(dtype, B=1, T=kv_len, D=D, q_len=q_len)
    q, k, v = w.qkv()
    bm = fa.block_mask("sink_window", 1, 1, q_len, kv_len, window=window, sinks=sinks)
    o, lse = fa.fwd(*parity.to_device(w, q, k, v), bm)
    fa.default_workspace("cuda").check()
    ro, rl = oracle.fwd(q, k, v, **_okw(window, sinks))
    parity.compare(o.double().cpu().numpy(), ro, lse.double().cpu().numpy(), rl, dtype, label="sinks")


@gpu
@pytest.mark.parametrize("score,skw", SCORES)
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("fp32", 128)])
def test_forward_scores(fa, dtype, D, score, skw):
    w = _case(dtype, T=500, D=D, score=score, **skw)
    q, k, v = w.qkv()
    bm = fa.block_mask("sink_window", 1, 1, 500, 500, window=70, sinks=5)
    o, lse = fa.fwd(*parity.to_device(w, q, k, v), bm, **parity.score_kwargs_gpu(w))
    fa.default_workspace("cuda").check()
    ro, rl = oracle.fwd(q, k, v, **_okw(70, 5), **parity.score_kwargs_oracle(w))
    parity.compare(o.double().cpu().numpy(), ro, lse.double().cpu().numpy(), rl, dtype, label=score)


@gpu
@pytest.mark.parametrize("q_len,kv_len,window,sinks", [(3, 700, 1, 1), (4, 2, 0, 1), (100, 130, 30, 4)])
def test_decode(fa, q_len, kv_len, window, sinks):
    w = _case(B=1, Hq=2, Hkv=2, T=kv_len, q_len=min(q_len, 16))
    q, k, v = w.qkv()
    bm = fa.block_mask("sink_window", 1, 1, w.Tq, kv_len, window=window, sinks=sinks)
    o, lse = fa.fwd_decode(*parity.to_device(w, q, k, v), bm)
    fa.default_workspace("cuda").check()
    ro, rl = oracle.fwd(q, k, v, **_okw(window, sinks))
    parity.compare(o.double().cpu().numpy(), ro, lse.double().cpu().numpy(), rl, "bf16", label="decode")


@gpu
@pytest.mark.parametrize("score,skw", SCORES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len,kv_len,window,sinks", [(300, 300, 40, 4), (520, 520, 128, 130), (1, 1, 0, 0),
                                                       (150, 420, 200, 30), (420, 150, 60, 2)])
def test_backward(fa, score, skw, D, q_len, kv_len, window, sinks):
    import torch
    w = _case(B=1, T=kv_len, D=D, q_len=q_len, score=score, **skw)
    q, k, v = w.qkv()
    g = synth.round_to_bf16(synth.standard_normal(78, q.shape))
    qd, kd, vd = parity.to_device(w, q, k, v)
    gd = torch.from_numpy(g).cuda().to(torch.bfloat16)
    bm = fa.block_mask("sink_window", 1, 1, q_len, kv_len, window=window, sinks=sinks)
    kw = parity.score_kwargs_gpu(w)
    o, lse = fa.fwd(qd, kd, vd, bm, **kw)
    grads = fa.bwd(qd, kd, vd, o, lse, gd, bm, **kw)
    fa.default_workspace("cuda").check()
    refs = oracle.bwd(q, k, v, g, **_okw(window, sinks), **parity.score_kwargs_oracle(w))
    for name, got, ref in zip(("dq", "dk", "dv"), grads, refs):
        err = np.abs(got.double().cpu().numpy() - ref)
        assert err.max() <= 2e-2 * max(1.0, np.abs(ref).max()), name
        norm = np.linalg.norm(ref)
        assert norm == 0 or np.linalg.norm(err) <= 1e-2 * norm, name


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,q_len,kv_len,window,sinks", [
    (1, 4, 2, 2000, 2000, 60, 4), (2, 2, 2, 1300, 1300, 10, 300), (1, 6, 1, 1100, 1100, 300, 129),
    (1, 2, 1, 3000, 200, 0, 150), (1, 3, 3, 900, 2000, 5, 1000), (1, 2, 2, 1500, 1500, 100, 2**31 - 1)])
def test_backward_with_split_sinks(fa, D, B, Hq, Hkv, q_len, kv_len, window, sinks):
    """Many more q-blocks than the window spans: the sinks' kv blocks are shared by several units, whose partial sums
    are added in order, so that two runs agree to the bit."""
    import torch
    w = _case(B=B, Hq=Hq, Hkv=Hkv, T=kv_len, D=D, q_len=q_len)
    q, k, v = w.qkv()
    g = synth.round_to_bf16(synth.standard_normal(79, q.shape))
    qd, kd, vd = parity.to_device(w, q, k, v)
    gd = torch.from_numpy(g).cuda().to(torch.bfloat16)
    bm = fa.block_mask("sink_window", 1, 1, q_len, kv_len, window=window, sinks=sinks)
    o, lse = fa.fwd(qd, kd, vd, bm)
    grads = fa.bwd(qd, kd, vd, o, lse, gd, bm)
    again = fa.bwd(qd, kd, vd, o, lse, gd, bm)
    fa.default_workspace("cuda").check()
    refs = oracle.bwd(q, k, v, g, **_okw(window, sinks))
    for name, got, twice, ref in zip(("dq", "dk", "dv"), grads, again, refs):
        assert torch.equal(got, twice), name
        err = np.abs(got.double().cpu().numpy() - ref)
        assert err.max() <= 2e-2 * max(1.0, np.abs(ref).max()), name
        assert np.linalg.norm(err) <= 1e-2 * np.linalg.norm(ref), name


def score_and_slope(x, i, j, score, softcap=1.0, slopes=None, rel_bias=None, rel_max=0):
    """The modified score and its derivative by the scaled one."""
    slope = np.ones_like(x)
    if slopes is not None:
        x = x - np.asarray(slopes, np.float64)[:, None, None] * np.abs(i - j)
    if "softcap" in score:
        t = np.tanh(x / softcap)
        x, slope = softcap * t, 1 - t * t
    if rel_bias is not None:
        x = x + np.asarray(rel_bias, np.float64)[:, np.clip(i - j, -rel_max, rel_max) + rel_max]
    return x, slope


@gpu
@pytest.mark.parametrize("score,skw", SCORES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len,kv_len,window,sinks", [(2, 2, 1, 0), (2, 2, 9, 0), (3, 3, 1, 1), (8, 8, 8, 0), (200, 200, 1, 0),
                                                       (200, 200, 3, 3), (300, 300, 0, 2), (140, 40, 5, 1), (9, 300, 100, 4), (300, 300, 11, 4), (20, 20, 30, 0),
                                                       (300, 300, 15, 0), (200, 200, 16, 0)])
def test_backward_of_few_keys(fa, score, skw, D, q_len, kv_len, window, sinks):
    """With few keys dP - Delta is small beside dP.  What may be off, element by element: the rounding of P and dS to
    bf16 (half a step, 2^-8 of each; the gradients are fp32); the soft-cap's tanh by 2.3e-5 of itself, which is
    2^-13 of P at a cap of 5 and 2^-14 of dS before its slope; and, of fp32 sums, 2^-15 of P (|dP| + |Delta|)."""
    import torch
    w = _case(B=1, Hq=4, Hkv=2, T=kv_len, D=D, q_len=q_len, score=score, **skw)
    q, k, v = w.qkv()
    g = synth.round_to_bf16(synth.standard_normal(80, q.shape))
    qd, kd, vd = parity.to_device(w, q, k, v)
    gd = torch.from_numpy(g).cuda().to(torch.bfloat16)
    bm = fa.block_mask("sink_window", 1, 1, q_len, kv_len, window=window, sinks=sinks)
    kw = parity.score_kwargs_gpu(w)
    o, lse = fa.fwd(qd, kd, vd, bm, **kw)
    grads = fa.bwd(qd, kd, vd, o, lse, gd, bm, **kw)
    fa.default_workspace("cuda").check()
    refs = oracle.bwd(q, k, v, g, **_okw(window, sinks), **parity.score_kwargs_oracle(w))
    # |dS|, P and the rest of the bounds, from the oracle's lse under the same score
    see, scale = dense(q_len, kv_len, window, sinks), 1 / np.sqrt(D)
    k2, v2 = (np.repeat(x, 2, 1).astype(np.float64) for x in (k, v))
    q2, g2 = q.astype(np.float64), g.astype(np.float64)
    x = q2 @ k2.swapaxes(-1, -2) * scale
    i, j = np.arange(q_len)[:, None], np.arange(kv_len)[None]
    x, slope = score_and_slope(x, i, j, **parity.score_kwargs_oracle(w))
    x = np.where(see, x, -np.inf)
    m = x.max(-1, keepdims=True)
    p = np.exp(x - np.where(np.isfinite(m), m, 0))
    p /= np.maximum(p.sum(-1, keepdims=True), 1e-300)
    dp = g2 @ v2.swapaxes(-1, -2)
    delta = (p * dp).sum(-1, keepdims=True)
    rounding = 2.0 ** -8 + 2.0 ** -13
    slack = np.abs(p * (dp - delta)) * (slope * rounding + 2.0 ** -14) + p * (np.abs(dp) + np.abs(delta)) * 2.0 ** -15
    # a row of more than 16 keys has its Delta from the bf16 O: each O_d off by half a step, so Delta by at most
    # 2^-8 sum_d |dO_d O_d|
    many = see.sum(-1)[:, None] > 16
    slack += np.where(many, p * (np.abs(g2 * (p @ v2)).sum(-1, keepdims=True) * 2.0 ** -8), 0)
    pair = lambda t: t.reshape(1, 2, 2, *t.shape[2:]).sum(2)                        # noqa: E731
    bounds = (scale * slack @ np.abs(k2), pair(scale * slack.swapaxes(-1, -2) @ np.abs(q2)),
              pair((p * rounding).swapaxes(-1, -2) @ np.abs(g2)))
    for name, got, ref, bound in zip(("dq", "dk", "dv"), grads, refs, bounds):
        err = np.abs(got.double().cpu().numpy() - ref)
        assert (err <= bound + 1e-6).all(), f"{name}: {(err / (bound + 1e-6)).max():.2f} of what it may be off"
