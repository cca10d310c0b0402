"""Soft-caps of the paged forward far above the scores, and far below them.

A cap C turns a score s into C tanh(s / C).  For C far above |s| that is s
itself, so its error has to go by s and not by C: tolerances are those of
tests/test_paged.py (scores up to 60 off by at most 4e-4), whatever the cap.
"""
import importlib.util
import os
import re

import numpy as np
import pytest
import torch

from tests.test_paged import Batch, compare, fa, reference, run  # noqa: F401  (fa: the fixture)

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_fa_gb300", "csrc")
gpu = pytest.mark.gpu


def _header():
    text = open(os.path.join(CSRC, "tanh_fine_poly.h")).read()
    return ([float(v) for v in re.findall(r"kTanhFineC\d = ([-0-9.e]+)f;", text)],
            float(re.search(r"kTanhFineRange = ([-0-9.e]+)f;", text).group(1)))


def test_header_matches_derivation():
    spec = importlib.util.spec_from_file_location("gen_poly", os.path.join(CSRC, "gen_poly.py"))
    g = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(g)
    c, err = g.tanh_coeffs(g.TANH_FINE_DEGREE, g.TANH_FINE_RANGE)
    hc, U = _header()
    assert U == g.TANH_FINE_RANGE
    np.testing.assert_allclose(hc, np.float32(c), rtol=0, atol=1e-7)
    assert err < 6e-7


@pytest.mark.parametrize("cap", [1e-3, 2.0, 50.0, 1e3, 1e5, 1e8, 1e30, 3e38])
def test_polynomial_as_the_kernels_fold_it(cap):
    """x mul q((x in)^2) in fp32: 5.7e-7 of the polynomial; half a step (6e-8) each for the last Horner step, the last
    two products and mul; what in, u, w and the steps before it add weighs at most a third of that: under 1e-6 of the
    score for every cap."""
    c, U = _header()
    f = np.float32
    big = np.finfo(f).max
    cin, mul = min(f(1) / f(cap), big), f(1.4426950408889634)
    x = (np.linspace(-U, U, 20001) * min(cap, 1e30)).astype(f)
    u = (x * cin).astype(f)
    w = (u * u).astype(f)
    q = np.full_like(w, c[-1])
    for k in c[-2::-1]:
        q = (q.astype(np.float64) * w + f(k)).astype(f)
    got = (x * mul).astype(f).astype(np.float64) * q
    want = cap * np.tanh(x.astype(np.float64) / f(cap)) * 1.4426950408889634
    assert (np.abs(got - want) <= 1e-6 * np.abs(want)).all()


@gpu
@pytest.mark.parametrize("q_scale", [0.1, 1.0, 8.0])
@pytest.mark.parametrize("cap", [1e-3, 1e3, 1e5, 1e8, 1e30, 3e38])
@pytest.mark.parametrize("score", ["softcap", "alibi_softcap"])
@pytest.mark.parametrize("n", [1, 40])
def test_caps(fa, n, score, cap, q_scale):  # noqa: F811
    kw = dict(slopes=np.random.default_rng(3).random(8).astype(np.float32) * 0.3) if score == "alibi_softcap" else {}
    run(fa, Batch([n] * 3, [n + 300, n + 90, n + 1000], 2, 64, 32), 8, score=score, softcap=cap, q_scale=q_scale, **kw)


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("score", ["softcap", "alibi_softcap"])
@pytest.mark.parametrize("shared", [0, 64])
@pytest.mark.parametrize("n", [2, 40])
def test_rows_past_the_cap_beside_rows_far_below_it(fa, n, shared, score, D):  # noqa: F811
    """Every other token's scores are a million times its neighbours': those rows are past the cap, and what the
    others get does not depend on it."""
    cap = 1e5
    bt = Batch([n] * 3, [shared + n + 300, shared + n + 90, shared + n + 1000], 2, D, 32, shared=shared)
    q = bt.queries(8)
    q[1::2] *= 2.0 ** 20
    kw = dict(slopes=np.random.default_rng(3).random(8).astype(np.float32) * 0.3) if score == "alibi_softcap" else {}
    gkw = {"alibi_slopes": torch.from_numpy(kw["slopes"]).cuda()} if kw else {}
    got = fa.fwd_paged(torch.from_numpy(q).cuda().to(torch.bfloat16), *bt.device(), max_q_len=n, shared_len=shared,
                       score=score, softcap=cap, **gkw)
    fa.default_workspace("cuda").check()
    o, lse, A = reference(bt, q, "causal", 0, 0, score, softcap=cap, **kw)
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
    o[1::2], lse[1::2] = np.nan, np.nan
    compare(got, (o, lse, A))
