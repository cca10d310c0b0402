"""What the cache held in 8 bits keeps of small shares: keys far below the largest
score, pages whose scales are far apart, sums over keys whose scales grow.

A key's share is 2^(its score in base 2) x (its page's v scale): what it adds to O,
for a code of 1.  The scores here are products of few bits (one element of q and k
is not 0), so that they are exact but for the fp32 scales: at most 8 roundings of
2^-24 on numbers below 256, 2^-13 in the exponent, and ex2.approx's 2^-22.

Tolerances, per column.  P is rounded to f16 at up to 2^15, and its reference lies
at least 2^8 of that below the largest share (where P takes v's scale with it), or 2^15
below the largest 2^score (9 to 16 rows, where it does not): half a step is 2^-11 of
the share, or, of the largest, 2^-25 / 2^8 = 2^-33 (2^-25 / 2^15 = 2^-40, times the
key's own v scale).  With w the exact weights and c the codes
     |O - exact| <= sum_j max(2^-11 share_j, floor_j) |c_j| / sum 2^score + 2^-12 sum_j w_j |v_j|,
the last for the exponent (2^-13 ln 2) and for fp32 sums (chains of at most 300 parts
and 64 products: 2^-15).  lse: 2^-13 ln 2 and 2^-15 of its sum.
"""
import functools

import numpy as np
import pytest
import torch

from tests.test_paged import fa  # noqa: F401  (the fixture)
from tests.test_paged_scaled import codes_of, e4m3

gpu = pytest.mark.gpu
PAGE = 64


@functools.lru_cache(4)
def uniform_codes(seed, shape):
    return e4m3(np.random.default_rng(seed).uniform(-0.2, 1.0, shape) * 448)


def codes(seed, shape):
    """e4m3 numbers, most of them of the last binades, with a mean that is not 0."""
    return uniform_codes(seed, shape).copy()


class Keys:
    """B sequences of n keys each of one kv head, a page after the other; scores[j] = k_codes[j] k_scale q0 / 16."""

    def __init__(self, B, k_code, k_scale, v_code, v_scale, D):
        # k_code [n], k_scale and v_scale [pages], v_code [n, D]: the same for every sequence
        self.B, self.D, self.n = B, D, len(k_code)
        pages = self.n // PAGE
        assert pages * PAGE == self.n
        self.k_code, self.k_scale, self.v_code, self.v_scale = k_code, k_scale.astype(np.float32), v_code, v_scale.astype(np.float32)
        k = np.zeros((pages, 1, PAGE, D))
        k[:, 0, :, 0] = k_code.reshape(pages, PAGE)
        each = lambda x: torch.cat([x] * B)     # noqa: E731
        self.kc = each(codes_of(k).cuda().view(torch.uint8)).view(torch.float8_e4m3fn)
        self.vc = each(codes_of(v_code.reshape(pages, 1, PAGE, D)).cuda().view(torch.uint8)).view(torch.float8_e4m3fn)
        s = lambda x: each(torch.from_numpy(x.astype(np.float32)).cuda()[:, None]).contiguous()     # noqa: E731
        self.scales = dict(k_scale=s(k_scale), v_scale=s(v_scale))
        self.table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
        self.kv = torch.full((B,), self.n, dtype=torch.int32, device="cuda")

    def run(self, fa, rows, shared=0, out_fp32=True):  # noqa: F811
        """`rows` query heads of one token per sequence (n = 1), q0 a little more from row to row."""
        q0 = 16 + np.arange(rows) * 0.125
        q = torch.zeros((self.B, rows, self.D), dtype=torch.bfloat16, device="cuda")
        q[..., 0] = torch.from_numpy(q0).cuda().to(torch.bfloat16)
        starts = torch.arange(self.B + 1, dtype=torch.int32, device="cuda")
        table = self.table
        if shared:
            table = table.clone()
            table[:, :shared // PAGE] = self.table[0, :shared // PAGE]
        o, lse = fa.fwd_paged(q, self.kc, self.vc, table, self.kv, starts, **self.scales, max_q_len=1, mask="full",
                              shared_len=shared, scale=1 / 16, out_fp32=out_fp32)
        fa.default_workspace("cuda").check()
        return o.double().cpu().numpy(), lse.double().cpu().numpy(), q0

    def check(self, got, rows, few, bf16_out=False):
        """few: P without v's scale (9 to 16 rows and no prefix)."""
        o, lse, q0 = got
        assert np.isfinite(o).all() and np.isfinite(lse).all()
        ks, vs = (np.repeat(x.astype(np.float64), PAGE) for x in (self.k_scale, self.v_scale))
        for r in range(rows):
            score = q0[r] / 16 * self.k_code * ks
            p = np.exp(score - score.max())
            total = p.sum()
            share = p * vs
            floor = 2.0 ** -40 * vs if few else 2.0 ** -33 * share.max()
            if 8 < rows <= 16:                   # (a prefix's part of the keys, and the others)
                floor = np.maximum(floor, 2.0 ** -40 * vs)
            ro, A = (p * vs) @ self.v_code / total, (p * vs) @ np.abs(self.v_code) / total
            tol = np.maximum(2.0 ** -11 * share, floor) @ np.abs(self.v_code) / total + 2.0 ** -12 * A
            if bf16_out:
                tol = tol + 2.0 ** -8 * np.abs(ro)
            err = np.abs(o[:, r] - ro)
            assert (err <= tol).all(), f"row {r}: o off by {np.nanmax(err / np.maximum(tol, 1e-300)):.2f} of what it may"
            rl = np.log(total) + score.max()
            assert np.abs(lse[:, r] - rl).max() <= 2.0 ** -13, f"row {r}: lse off by {np.abs(lse[:, r] - rl).max()}"


# rows per kv head, and what a prefix of half the keys makes of them: every kernel
KERNELS = [(4, False), (12, False), (40, False), (4, True), (12, True), (40, True)]


def few(rows, shared):
    return 8 < rows <= 16 and not shared


@gpu
@pytest.mark.parametrize("rows,prefix", KERNELS)
@pytest.mark.parametrize("nats", [17, 18, 20])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("B,n", [(1, 1 << 15), (300, 1 << 12)])
def test_a_sink_of_small_value(fa, rows, prefix, nats, D, first, B, n):  # noqa: F811
    """One key with a value of 0 far above all others, which are all of O (one sequence: over all CTAs, a part of it
    to each; many: a sequence or so to each)."""
    k = np.full(n, -256.0)
    v = codes(1, (n, D))
    sink = 5 if first else n - 3
    k[sink], v[sink] = 0.0, 0.0
    r = np.random.default_rng(nats)
    bt = Keys(B, k, nats / 256.0 * r.uniform(0.98, 1.0, n // PAGE), v, 2.0 ** -9 * r.uniform(0.7, 1.4, n // PAGE), D)
    shared = n // 2 if prefix else 0
    bt.check(bt.run(fa, rows, shared), rows, few(rows, prefix))


@gpu
@pytest.mark.parametrize("rows,prefix", KERNELS)
@pytest.mark.parametrize("apart", [12, 20, 24, 30])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [1, 40])
def test_columns_that_only_small_pages_have(fa, rows, prefix, apart, D, B):  # noqa: F811
    """Pages whose v scales are 2^apart of the others', which are 0 in the even columns."""
    n = 2048
    r = np.random.default_rng(apart)
    large = r.permutation(n // PAGE) < 8
    v = codes(2, (n, D))
    v[np.repeat(large, PAGE)[:, None] & (np.arange(D) % 2 == 0)] = 0.0
    bt = Keys(B, e4m3(r.uniform(-40, 0, n)), r.uniform(0.02, 0.03, n // PAGE), v,
              np.where(large, 1.0, 2.0 ** -apart) * r.uniform(0.7, 1.0, n // PAGE), D)
    bt.check(bt.run(fa, rows, n // 2 if prefix else 0), rows, few(rows, prefix))


@gpu
@pytest.mark.parametrize("rows,prefix", KERNELS)
@pytest.mark.parametrize("D", [64, 128])
def test_the_same_in_bf16(fa, rows, prefix, D):  # noqa: F811
    """As above with an output of 16 bits, where the running maximum may be passed."""
    n, r = 4096, np.random.default_rng(3)
    k = e4m3(-256 * r.uniform(0, 1, n))
    bt = Keys(3, np.sort(k), np.full(n // PAGE, 20 / 256.0), codes(5, (n, D)),
              2.0 ** r.integers(-20, 1, n // PAGE), D)
    bt.check(bt.run(fa, rows, n // 2 if prefix else 0, out_fp32=False), rows, few(rows, prefix), bf16_out=True)


@gpu
@pytest.mark.parametrize("rows,prefix", KERNELS)
@pytest.mark.parametrize("small,large", [(0.0, 2.0 ** 20), (0.0, 2.0 ** 100), (2.0 ** -100, 2.0 ** 60), (2.0 ** -60, 2.0 ** 100)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,n", [(1, 256), (1, 8192), (160, 512)])
@pytest.mark.parametrize("order", ["grow", "shrink", "mixed"])
def test_scales_that_grow(fa, rows, prefix, small, large, D, B, n, order):  # noqa: F811
    """Pages with v scales of 0 or nearly that, then large ones: lse is that of all keys, and O over it."""
    r = np.random.default_rng(n)
    at = np.arange(n // PAGE) < n // PAGE // 2
    at = {"grow": at, "shrink": ~at, "mixed": r.permutation(at)}[order]
    bt = Keys(B, e4m3(r.uniform(-40, 0, n)), r.uniform(0.02, 0.03, n // PAGE), codes(4, (n, D)),
              np.where(at, small, large * r.uniform(0.7, 1.0, n // PAGE)), D)
    bt.check(bt.run(fa, rows, n // 2 if prefix else 0), rows, few(rows, prefix))


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [False, True])
def test_elements_of_q_far_below_the_row_s_largest(fa, D, prefix):  # noqa: F811
    """In the kernel for many rows, and for a prefix with any, q is the sum of two e4m3 numbers, a row's largest element at
    224 to 448 of their units: exact down to 2^-2 of a unit, 2^-9.8 of the largest, and off by half of lo's least step,
    2^-10 of a unit or 2^-17.8 of the largest, below.  One key whose first element is 0 and whose second is 448: its score
    is lse, q1 x 448 / 16 but for fp32's 4 roundings."""
    Hq, r = 64, np.random.default_rng(1)
    q = np.zeros((1, Hq, D))
    q[0, :, 0] = r.choice([225 / 256, 226 / 256, 1.0, 1.25, 1.75, 447 / 256 - 1 / 256], Hq)
    q[0, :, 1] = 2.0 ** -r.integers(8, 20, Hq) * r.integers(128, 256, Hq) / 128
    q[0, ::7, 1] = 255 / 256 / 1024              # the largest that the split may miss
    q[0, 1::7, 1] = 2.0 ** -9                    # and one that it holds
    qd = torch.from_numpy(q).cuda().to(torch.bfloat16)
    assert (qd.double().cpu().numpy() == q).all()
    pages = 2 if prefix else 1
    k = torch.zeros((pages, 1, PAGE, D), device="cuda")
    k[..., 1] = 448
    v = torch.ones((pages, 1, PAGE, D), device="cuda")
    one = torch.ones((pages, 1), device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")     # noqa: E731
    n = PAGE + 1 if prefix else 1
    f8 = torch.float8_e4m3fn
    o, lse = fa.fwd_paged(qd, k.to(f8), v.to(f8), i32(*range(pages)).view(1, -1), i32(n), i32(0, 1), k_scale=one, v_scale=one.clone(),
                          max_q_len=1, mask="full", shared_len=PAGE if prefix else 0, scale=1 / 16, out_fp32=True)
    fa.default_workspace("cuda").check()
    top, score = q[0, :, 0], q[0, :, 1] * 448 / 16
    off = np.abs(lse.double().cpu().numpy()[0] - score - np.log(n))
    exact = q[0, :, 1] >= 2.0 ** -9 * top
    # (lse itself is rounded, and the prefix's products are summed: 2^-20)
    assert exact.any() and (off[exact] <= 2.0 ** -20 * 8).all()
    assert (~exact).any() and (off[~exact] <= 2.0 ** -17.8 * (top * 448 / 16)[~exact] + 2.0 ** -17).all()
    assert torch.allclose(o.float(), torch.ones_like(o.float()), atol=1e-6)


@gpu
@pytest.mark.parametrize("rows,prefix,power", [(rows, False, power) for rows in (4, 12)
                                               for power in (20, 23, 24, 25, 26, 27, 28, 30, 34)]
                         + [(40, prefix, power) for prefix in (False, True) for power in (20, 22, 23)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("B", [3, 400])
def test_scores_past_20_bits(fa, rows, prefix, power, sign, B):  # noqa: F811
    """Scores so large that a reference 8 or 15 below them is rounded, by up to 16: all are the same, so that O is the mean.
    (P may end up at 2^16, which f16 ends just below: 2^-11 of O.  In the kernel for many rows the product of S and its
    scale is not rounded but the reference is, by half a unit of scores past 2^23, and P may be anything beyond.)"""
    n, D = 512, 64
    bt = Keys(B, np.full(n, sign * 256.0), np.full(n // PAGE, 2.0 ** (power - 8)), codes(6, (n, D)), np.ones(n // PAGE), D)
    o, lse, q0 = bt.run(fa, rows, n // 2 if prefix else 0)
    assert np.isfinite(o).all() and np.isfinite(lse).all()
    mean, A = bt.v_code.mean(0), np.abs(bt.v_code).mean(0)
    assert (np.abs(o - mean) <= (2.0 ** -10 + 2.0 ** -12) * A).all()
    score = q0 * sign * 2.0 ** (power - 4)
    assert (np.abs(lse - (score + np.log(n))) <= np.abs(score) * 2.0 ** -21 + 2.0 ** -13).all()
