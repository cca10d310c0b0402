"""Windows wider than any sequence, up to the largest 32-bit number: the mask is
the causal one, forward and backward."""
import numpy as np
import pytest

import oracle
from block_sparse_attention_fa_gb300 import synth
from tests import parity

pytestmark = pytest.mark.gpu

SIZES = [(300, 300), (130, 400), (400, 130), (17, 17)]
WINDOWS = [2**31 - 1, 2**31 - 100, 2**31 - 400]


def _step(mask, q_len, kv_len, D, **mkw):
    import torch
    from block_sparse_attention_fa_gb300 import fa
    w = synth.Workload(name="wide", dtype="bf16", B=1, Hq=4, Hkv=2, T=kv_len, D=D, mask="causal", seed=62, q_len=q_len)
    q, k, v = w.qkv()
    g = synth.round_to_bf16(synth.standard_normal(81, q.shape))
    x = parity.to_device(w, q, k, v)
    bm = fa.block_mask(mask, 1, 1, q_len, kv_len, **mkw)
    o, lse = fa.fwd(*x, bm)
    grads = fa.bwd(*x, o, lse, torch.from_numpy(g).cuda().to(torch.bfloat16), bm)
    fa.default_workspace("cuda").check()
    return (o, lse, *grads), (q, k, v, g)


@pytest.mark.parametrize("q_len,kv_len", SIZES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", WINDOWS)
def test_sliding_window_is_causal(window, D, q_len, kv_len):
    """One mask, one order of sums: the same bits."""
    import torch
    got, _ = _step("sliding_window", q_len, kv_len, D, window=window)
    want, _ = _step("causal", q_len, kv_len, D)
    for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), got, want):
        assert torch.equal(a, b), name


@pytest.mark.parametrize("q_len,kv_len", SIZES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", WINDOWS)
def test_sink_window_gradients(window, D, q_len, kv_len):
    """Against the oracle, to the backward's tolerances (tests/test_bwd_gpu.py): Delta of rows with few keys is
    another sum here."""
    got, x = _step("sink_window", q_len, kv_len, D, window=window, sinks=3)
    for name, a, ref in zip(("dq", "dk", "dv"), got[2:], oracle.bwd(*x, mask="causal")):
        err = np.abs(a.double().cpu().numpy() - ref)
        assert err.max() <= 2e-2 * max(1.0, np.abs(ref).max()), name
        assert np.linalg.norm(err) <= 1e-2 * np.linalg.norm(ref), name
