"""The paged cache held in 8 bits (fa_kv_append_scaled, fa_fwd_paged_scaled)
against plain float64 forms.

Tolerances, derived:
  forward  A code and a bf16 number are exact in f16 (a row of q scaled by a power
       of two; elements 2^28 below its largest lose less than 2^-39 of that), so
       the products are exact and the sums fp32's; the scales are two more fp32
       roundings.  In larger units (more than 16 rows per sequence and kv head, or
       a shared prefix) q is the sum of two e4m3 numbers: exact down to 2^-10 of a
       row's largest element, 2^-18 of that off below, so that a score is off by
       2^-18 max|q| sum|k| scale at most (below 1e-6 for normal q and k, of which 1
       element in 400 is that small).  The scores' error, with ex2.approx and a
       soft-cap in fp32, stays below 4e-4 in the exponent for |s| <= 60, as for the
       bf16 cache.
       P is rounded to f16: half a step is 2^-11 of p, or 2^-25 below 2^-14 (P is
       relative to a share that one of the keys has in O, v's scale included).  With
       A = sum_j w_j |v_j| and V the largest |v| the output is off by at most
       (2^-11 + 4e-4) A + 2^-25 n V; the output's own rounding adds 2^-8 |o| (bf16),
       and fp32 sums of O 1e-5 of the larger of 1 and V.
  lse  the scores' error, 4e-4.
  append   A code is off by at most half a step of e4m3 at |x / scale|
       (2^-4 of its binade, 2^-10 below 2^-6) and by the fp32 rotation, 3 roundings
       of 2^-24 on |x0 c| + |x1 s|.  Scales and codes rounded again are powers of
       two and roundings of numbers that fp32 holds: exact.
"""
import ctypes

import numpy as np
import pytest
import torch

from block_sparse_attention_fa_gb300 import synth
from tests.test_paged import (FAKE, MASKS, SCORES, Batch, _append, _fwd, _kv, fa, reference,  # noqa: F401
                              score_kw)

gpu = pytest.mark.gpu
E4M3_MAX = 448.0


def e4m3(y):
    """The nearest e4m3 numbers, ties to even, in float64."""
    a = np.minimum(np.abs(y), E4M3_MAX)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.copysign(np.minimum(np.round(a / step) * step, E4M3_MAX), y)


def half_step(y):
    return 2.0 ** (np.floor(np.log2(np.clip(np.abs(y), 2.0 ** -6, E4M3_MAX))) - 4)


def least_scale(amax):
    """The smallest power of two s, 2^-100 .. 2^119, with amax <= 448 s."""
    e = -100
    while amax > E4M3_MAX * 2.0 ** e and e < 119:
        e += 1
    return 2.0 ** e


def codes_of(x):
    """A float array as e4m3 codes (NaN stays NaN)."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.float8_e4m3fn)


class Batch8(Batch):
    """A Batch whose cache is held in 8 bits: scales `kind` pow2 or any, of pages that no sequence has NaN."""

    def __init__(self, *a, kind="pow2", spread=1.0, **kw):
        super().__init__(*a, **kw)
        r = np.random.default_rng(len(self.new) + self.page)
        n = self.kc.shape[:2]
        owned = np.zeros(n[0], bool)
        for b, L in enumerate(self.kv):
            owned[self.table[b, :-(-L // self.page)]] = True
        for name, values in (("k", self.kc), ("v", self.vc)):
            scale = 2.0 ** np.round(r.normal(-6.5, spread, n))
            if kind == "any":
                scale = scale * r.uniform(0.7, 1.4, n)
            if self.shared % self.page:          # the prefix's last keys, in common as values: copied with their scale
                last = self.table[:, self.shared // self.page]
                scale[last[last >= 0]] = scale[self.table[0, self.shared // self.page]]
            scale = np.where(owned[:, None], scale, np.nan).astype(np.float32)
            with np.errstate(invalid="ignore"):
                y = values / scale[:, :, None, None]
            codes = np.where(np.isnan(y), np.nan, e4m3(np.nan_to_num(y)))
            setattr(self, name + "_codes", codes)
            setattr(self, name + "_scale", scale)
            real = codes * scale[:, :, None, None].astype(np.float64)
            rows = getattr(self, name)
            for b, L in enumerate(self.kv):
                j = np.arange(L)
                rows[b] = real[self.table[b, j // self.page], :, j % self.page]

    def device8(self):
        kc, vc, table, kv, qs = self.device()
        f = lambda x: torch.from_numpy(x).cuda()   # noqa: E731
        return (codes_of(self.k_codes).cuda(), codes_of(self.v_codes).cuda(), table, kv, qs), \
            dict(k_scale=f(self.k_scale), v_scale=f(self.v_scale))


def compare8(got, ref, bt, bf16_out=True, score_err=0.0):
    """score_err [rows, heads]: what the scores may be off by beside 4e-4."""
    (o, lse), (ro, rl, A) = got, ref
    more = np.broadcast_to(score_err, rl.shape)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    rows = ~np.isnan(rl)
    V = max([np.abs(v).max() for v in bt.v if v.size] + [0.0])
    tol = (2.0 ** -11 + 4e-4 + 2 * more[..., None]) * A + 2.0 ** -25 * max(bt.kv) * V \
        + (2.0 ** -8 * np.abs(ro) if bf16_out else 0) + 1e-5 * max(V, 1)
    assert np.isfinite(o[rows]).all()
    err = np.abs(o - ro)[rows]
    assert (err <= tol[rows]).all(), f"o off by {np.nanmax(err / tol[rows]):.2f} of what it may"
    assert (np.abs(lse - rl) <= 4e-4 + more)[rows].all(), f"lse off by {np.nanmax(np.abs(lse - rl)[rows])}"


def run8(fa, bt, Hq, mask="causal", window=0, sinks=0, score="none", q_scale=1.0, out_fp32=False, scale=None,  # noqa: F811
         max_q_len=None, q=None, fused=False, score_err=0.0, **kw):
    q = bt.queries(Hq, scale=q_scale) if q is None else q
    dev, scales = bt.device8()
    qd = torch.from_numpy(q).cuda().to(torch.bfloat16)
    if fused:                                    # a slice of a projection's rows
        wide = torch.zeros((bt.total, Hq + 3, bt.D), dtype=torch.bfloat16, device="cuda")
        wide[:, 2:2 + Hq] = qd
        qd = wide[:, 2:2 + Hq]
    gkw = {}
    if "softcap" in kw:
        gkw["softcap"] = kw["softcap"]
    if "slopes" in kw:
        gkw["alibi_slopes"] = torch.from_numpy(kw["slopes"].astype(np.float32)).cuda()
    if "rel_bias" in kw:
        gkw.update(rel_bias=torch.from_numpy(kw["rel_bias"].astype(np.float32)).cuda().contiguous(), rel_max=kw["rel_max"])
    most = max_q_len or max(max(bt.new), 1)
    out = torch.full((bt.total, Hq, bt.D), 7.0, dtype=torch.float32 if out_fp32 else torch.bfloat16, device="cuda")
    got = fa.fwd_paged(qd, *dev, **scales, max_q_len=most, mask=mask, window=window, sinks=sinks, shared_len=bt.shared,
                       score=score, out_fp32=out_fp32, scale=scale, out=out,
                       lse=torch.full((bt.total, Hq), 7.0, device="cuda"), **gkw)
    fa.default_workspace("cuda").check()
    compare8(got, reference(bt, q, mask, window, sinks, score, scale, **kw), bt, not out_fp32, score_err)
    for x in got:                                # rows behind the last sequence
        assert (x[int(bt.q_start[-1]):] == 7).all()
    return got


# ------------------------------------------------------------------ CPU: refusals
def _scales8(fa, **kw):  # noqa: F811
    s = fa.PagedScales(FAKE, FAKE + (1 << 20))
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw", [dict(k_scale=None), dict(v_scale=None), dict(k_scale=FAKE + 2), dict(v_scale=FAKE),
                                dict(v_scale=FAKE + 60), dict(k_scale=FAKE + (1 << 20) - 4)], ids=str)
def test_refused_scales(fa, kw):  # noqa: F811
    lib, c = fa.load_library(), _kv(fa, v=FAKE + (1 << 20))
    m, sc = fa.MaskDesc(), fa.ScoreDesc()
    m.kind = 1
    for s in (ctypes.byref(_scales8(fa, **kw)), None):
        assert lib.fa_kv_append_scaled(ctypes.byref(c), s, ctypes.byref(_append(fa)), FAKE, None) == fa.ERR_INVALID_ARG
        assert b"scale" in lib.fa_last_error()
        assert lib.fa_fwd_paged_scaled(ctypes.byref(c), s, ctypes.byref(_fwd(fa)), ctypes.byref(m), ctypes.byref(sc), FAKE,
                                       1 << 40, FAKE, None) == fa.ERR_INVALID_ARG
        assert b"scale" in lib.fa_last_error()


def test_scaled_calls_check_the_rest(fa):  # noqa: F811
    lib, s = fa.load_library(), _scales8(fa)
    m, sc = fa.MaskDesc(), fa.ScoreDesc()
    m.kind = 1

    def append(c=None, a=None):
        return lib.fa_kv_append_scaled(ctypes.byref(c or _kv(fa, v=FAKE + (1 << 20))), ctypes.byref(s),
                                       ctypes.byref(a or _append(fa)), FAKE, None)

    def fwd(c=None, a=None, n=1 << 40):
        return lib.fa_fwd_paged_scaled(ctypes.byref(c or _kv(fa, v=FAKE + (1 << 20))), ctypes.byref(s),
                                       ctypes.byref(a or _fwd(fa)), ctypes.byref(m), ctypes.byref(sc), FAKE, n, FAKE, None)

    for kw, st in ((dict(D=96), 2), (dict(page_size=24), 2), (dict(k=None), 1), (dict(v=FAKE + 8), 1), (dict(B=0), 1)):
        assert append(_kv(fa, **kw)) == fwd(_kv(fa, **kw)) == st
    # 8 pages x 2 heads x 16 tokens x 128 columns of one byte
    assert append(_kv(fa, v=FAKE + 32768 - 16)) == fa.ERR_INVALID_ARG and b"k and v overlap" in lib.fa_last_error()
    assert append(a=_append(fa, rot_dim=8)) == fa.ERR_UNSUPPORTED
    assert append(a=_append(fa, q_out_stride=(64, 128), q_stride=(64, 128))) == fa.ERR_INVALID_ARG
    assert fwd(a=_fwd(fa, Hq=3)) == fa.ERR_INVALID_ARG
    assert fwd(n=100) == fa.ERR_INVALID_ARG and b"scratch" in lib.fa_last_error()
    assert append(_kv(fa, total_q=0)) == fwd(_kv(fa, total_q=0)) == fa.OK
    assert fa._PAGED_SCALES.size == ctypes.sizeof(fa.PagedScales)


# ------------------------------------------------------------------ GPU: append
def turned(a, i, rot, interleaved, cos, sin):
    """a rotated to position i, and what the fp32 rotation may be off by (of 2^-24 x 3)."""
    a = a.astype(np.float64)
    y, mag = a.copy(), np.zeros_like(a)
    if rot:
        p0 = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
        p1 = p0 + 1 if interleaved else p0 + rot // 2
        c, s = cos[i].astype(np.float64), sin[i].astype(np.float64)
        y[..., p0], y[..., p1] = a[..., p0] * c - a[..., p1] * s, a[..., p0] * s + a[..., p1] * c
        mag[..., p0], mag[..., p1] = np.abs(a[..., p0] * c) + np.abs(a[..., p1] * s), \
            np.abs(a[..., p0] * s) + np.abs(a[..., p1] * c)
    return y, mag


def check_append(name, got, got_scale, codes0, scale0, rows, bt, page):
    """One of k, v after an append; rows[b] = (values [n, Hkv, D], their rotations' magnitude)."""
    got, got_scale = got.float().double().cpu().numpy(), got_scale.double().cpu().numpy()
    want, want_scale = codes0.copy(), scale0.astype(np.float64).copy()
    near = np.zeros(want.shape)                  # what a code may be off by (0: exact)
    for b, (n, L) in enumerate(zip(bt.new, bt.kv)):
        for e in range((L - n) // page, (L - 1) // page + 1) if n else ():
            pg, f, t = bt.table[b, e], max(e * page, L - n), min((e + 1) * page, L)
            x, mag = (z[f - (L - n): t - (L - n)] for z in rows[b])
            for h in range(bt.Hkv):
                a = np.abs(x[:, h])
                s = least_scale(a[np.isfinite(a)].max(initial=0.0))
                if f > e * page:
                    before = want_scale[pg, h]
                    s = max(s, before)
                    want[pg, h, :f - e * page] = e4m3(want[pg, h, :f - e * page] * (before / s))
                want_scale[pg, h] = s
                at = slice(f - e * page, t - e * page)
                y = x[:, h] / s
                want[pg, h, at] = np.where(np.isfinite(y), y, np.nan)
                near[pg, h, at] = np.where(np.isfinite(y), half_step(np.nan_to_num(y, posinf=0, neginf=0)), 0) \
                    + 3 * 2.0 ** -24 * mag[:, h] / s
    assert np.array_equal(got_scale, want_scale, equal_nan=True), name
    nan = np.isnan(want)
    assert np.array_equal(nan, np.isnan(got)), name
    sat = np.clip(want, -E4M3_MAX, E4M3_MAX)
    assert (np.abs(got - sat)[~nan] <= near[~nan] * (1 + 1e-12)).all(), name


def run_append(fa, bt, x, Hq, rot, interleaved, cos, sin, fused=True):  # noqa: F811
    Hkv, T = bt.Hkv, bt.total
    (kc, vc, table, kv, qs), s = bt.device8()
    xd = torch.from_numpy(x).cuda().to(torch.bfloat16)
    q, k, v = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    kw = dict(cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda()) if rot else {}
    out = torch.full((T, Hq, bt.D), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.kv_append(q, k, v, kc, vc, table, kv, qs, **s, interleaved=interleaved, q_out=out, **kw)
    fa.default_workspace("cuda").check()
    rows = dict(k=[], v=[])
    got_q = out.double().cpu().numpy()
    for b, (n, L) in enumerate(zip(bt.new, bt.kv)):
        r0, ks = bt.q_start[b], []
        for t in range(n):
            y, mag = turned(x[r0 + t, :Hq], L - n + t, rot, interleaved, cos, sin)
            assert (np.abs(got_q[r0 + t] - y) <= np.where(mag > 0, 2.0 ** -8 * np.abs(y) + 3 * 2.0 ** -24 * mag, 0)).all()
            ks.append(turned(x[r0 + t, Hq:Hq + Hkv], L - n + t, rot, interleaved, cos, sin))
        rows["k"].append([np.array([z[e] for z in ks]).reshape(n, Hkv, bt.D) for e in range(2)])
        vs = x[r0:r0 + n, Hq + Hkv:].astype(np.float64)
        rows["v"].append([vs, np.zeros_like(vs)])
    assert (got_q[bt.q_start[-1]:] == 7).all()
    check_append("k", kc, s["k_scale"], bt.k_codes, bt.k_scale, rows["k"], bt, bt.page)
    check_append("v", vc, s["v_scale"], bt.v_codes, bt.v_scale, rows["v"], bt, bt.page)


def tables(n, rot):
    ang = np.random.default_rng(1).random((n, max(rot // 2, 1))) * 7
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


@gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 64, True), (64, 64, False), (64, 16, True),
                                               (128, 48, False), (64, 0, False), (128, 128, True)])
@pytest.mark.parametrize("fused", [True, False])
def test_append(fa, page, D, rot, interleaved, fused):  # noqa: F811
    bt = Batch8([1, 0, 5, 300, 2], [1, 7, 261, 300, 130], 2, D, page, pad=3)
    x = synth.round_to_bf16(synth.standard_normal(9, (bt.total, 10, D)))
    run_append(fa, bt, x, 6, rot, interleaved, *tables(301, rot), fused)


@gpu
@pytest.mark.parametrize("Hkv,B", [(1, 1), (3, 40), (8, 300), (16, 5)])
@pytest.mark.parametrize("page", [16, 128])
def test_append_single_tokens(fa, Hkv, B, page):  # noqa: F811
    r = np.random.default_rng(B)
    bt = Batch8([1] * B, list(r.integers(1, 400, B)), Hkv, 64, page, spread=3.0)
    x = synth.round_to_bf16(synth.standard_normal(9, (bt.total, 2 * Hkv + 2, 64)))
    run_append(fa, bt, x, 2, 32, False, *tables(401, 32))


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_append_sizes_of_values(fa, D):  # noqa: F811
    """Largest values at and around the borders of the scales, zeros, infinities, NaN, tiny and huge ones."""
    tops = [448.0, 450.0, 446.0, 7.0, 7.03125, 1.75, 1.7578125, 0.0, 2.0 ** -133, 2.0 ** -120, 3.3e38, 2.0 ** 127, 2.0 ** 120,
            1e-30, 0.5, 896.0]
    Hkv, n = len(tops), 5
    bt = Batch8([n, 2], [n, 40], Hkv, D, 16)
    r = np.random.default_rng(4)
    x = np.zeros((bt.total, 2 * Hkv + 1, D), np.float32)
    for h, top in enumerate(tops):
        z = r.uniform(-1, 1, (bt.total, D)) * top
        z[0, h % D] = top
        z[n, h % D] = -top
        x[:, 1 + h] = z
        x[:, 1 + Hkv + h] = z
    x = synth.round_to_bf16(x)
    x[1, 1 + 3, 5], x[2, 1 + Hkv + 3, 5], x[3, 1 + 4, 6] = np.inf, -np.inf, np.nan
    run_append(fa, bt, x, 1, 0, False, None, None)


@gpu
def test_append_grows_a_page(fa):  # noqa: F811
    """Single tokens, each larger than the ones before: earlier codes are rounded again with every step."""
    Hkv, D, page = 2, 64, 32
    kc = torch.zeros((2, Hkv, page, D), dtype=torch.float8_e4m3fn, device="cuda")
    vc, ks = kc.clone(), torch.full((2, Hkv), float("nan"), device="cuda")
    vs = ks.clone()
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    qs = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    x = synth.round_to_bf16(synth.standard_normal(3, (20, 2 * Hkv, D)))
    x *= 2.0 ** np.array([0, 0, 1, 1, 5, 0, 9, 9, 9, 2, 12, 0, 0, 20, 0, 0, 1, 2, 21, 0])[:, None, None]
    codes, scale = np.zeros((2 * Hkv, page, D)), np.zeros(2 * Hkv)
    for t in range(20):
        xd = torch.from_numpy(x[t:t + 1]).cuda().to(torch.bfloat16)
        fa.kv_append(None, xd[:, :Hkv], xd[:, Hkv:], kc, vc, table, torch.tensor([t + 1], dtype=torch.int32, device="cuda"),
                     qs, k_scale=ks, v_scale=vs)
        for h in range(2 * Hkv):
            s = max(least_scale(np.abs(x[t, h]).max()), scale[h])
            codes[h, :t] = e4m3(codes[h, :t] * (scale[h] / s))
            codes[h, t], scale[h] = e4m3(x[t, h] / s), s
        assert np.array_equal(torch.cat([ks[1], vs[1]]).cpu().numpy(), scale)
        got = torch.cat([kc[1].float(), vc[1].float()]).cpu().numpy()
        assert np.array_equal(got, codes)
    assert not kc[0].float().any() and ks[0].isnan().all()
    fa.default_workspace("cuda").check()


@gpu
def test_append_positions_outside_the_tables(fa):  # noqa: F811
    bt = Batch8([3, 2], [20, 40], 2, 64, 16)
    (kc, vc, table, kv, qs), s = bt.device8()
    x = torch.randn(5, 8, 64, device="cuda").to(torch.bfloat16)
    x[1] *= 1000                                 # its token is not written, and is not looked at
    ang = torch.rand(50, 32, device="cuda")
    pos = torch.tensor([4, 50, 49, 7, 7], dtype=torch.int32, device="cuda")
    before = kc.float().clone()
    fa.kv_append(x[:, :4], x[:, 4:6], x[:, 6:], kc, vc, table, kv, qs, **s, cos=ang.cos(), sin=ang.sin(), positions=pos)
    with pytest.raises(fa.FAError) as e:
        fa.default_workspace("cuda").check()
    assert e.value.status == fa.ERR_DEVICE_CHECK
    pg = bt.table[0, 1]
    want = before[pg, :, 2].cpu().numpy()
    old = torch.from_numpy(bt.k_scale[pg]).cuda()
    assert (s["k_scale"][pg] < 1000 * 4 / 448).all()
    want = e4m3(np.nan_to_num(want) * (old / s["k_scale"][pg])[:, None].cpu().numpy().astype(np.float64))
    assert np.array_equal(np.nan_to_num(kc[pg, :, 2].float().cpu().numpy()), want) or \
        np.array_equal(np.nan_to_num(kc[pg, :, 2].float().cpu().numpy()), np.nan_to_num(before[pg, :, 2].cpu().numpy()))


# ------------------------------------------------------------ GPU: single tokens
@gpu
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mask,window,sinks", MASKS)
def test_decode_masks(fa, page, D, mask, window, sinks):  # noqa: F811
    run8(fa, Batch8([1, 1, 1, 1, 1], [1, 700, 129, 128, 300], 2, D, page), 8, mask, window, sinks)


@gpu
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("out_fp32", [False, True])
def test_decode_scores(fa, score, D, out_fp32):  # noqa: F811
    run8(fa, Batch8([2, 1, 0, 3], [500, 40, 10, 333], 2, D, 16, kind="any"), 6, "sink_window", 200, 3, score=score,
         out_fp32=out_fp32, **score_kw(score, 6))


@gpu
@pytest.mark.parametrize("Hq,Hkv,n", [(1, 1, 1), (1, 1, 16), (16, 1, 1), (4, 4, 3), (9, 3, 5), (14, 2, 2), (5, 1, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_groups(fa, Hq, Hkv, n, D):  # noqa: F811
    r = np.random.default_rng(Hq)
    kv = list(r.integers(n, 600, 7))
    run8(fa, Batch8([n] * 6 + [max(n - 1, 1)], kv, Hkv, D, 32, kind="any", pad=2), Hq)


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
def test_decode_long_and_many(fa, D, page):  # noqa: F811
    run8(fa, Batch8([1, 1], [5000, 9000], 1, D, page, kind="any"), 4)
    r = np.random.default_rng(2)
    run8(fa, Batch8([1] * 700, list(r.integers(1, 90, 700)), 1, D, page), 2)


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_decode_scales_far_apart(fa, D):  # noqa: F811
    """Pages whose scales differ by many powers of two; queries of any size."""
    run8(fa, Batch8([1, 2], [300, 500], 2, D, 16, kind="any", spread=3.0), 4, q_scale=0.01)
    run8(fa, Batch8([1, 2], [300, 500], 2, D, 16), 4, q_scale=1e-30)
    run8(fa, Batch8([1, 2], [300, 500], 2, D, 16), 4, q_scale=1e6, scale=1e-7)


# ---------------------------------------------------------------- GPU: many rows
@gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mask,window,sinks", MASKS)
def test_chunk_masks(fa, page, D, mask, window, sinks):  # noqa: F811
    run8(fa, Batch8([100, 1, 40, 0, 130], [100, 700, 129, 10, 300], 2, D, page, pad=2), 8, mask, window, sinks)


@gpu
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("out_fp32", [False, True])
def test_chunk_scores(fa, score, D, out_fp32):  # noqa: F811
    run8(fa, Batch8([60, 1, 0, 33], [500, 40, 10, 333], 2, D, 32, kind="any"), 6, "sink_window", 200, 3, score=score,
         out_fp32=out_fp32, **score_kw(score, 6))


@gpu
@pytest.mark.parametrize("Hq,Hkv,n", [(1, 1, 17), (1, 1, 300), (3, 1, 90), (4, 4, 129), (16, 2, 7), (14, 2, 300)])
@pytest.mark.parametrize("D", [64, 128])
def test_chunk_groups(fa, Hq, Hkv, n, D):  # noqa: F811
    r = np.random.default_rng(Hq)
    kv = list(r.integers(n, n + 1200, 5))
    run8(fa, Batch8([n] * 4 + [n - 1], kv, Hkv, D, 64, kind="any", spread=2.0), Hq)


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_chunk_long_and_many(fa, D):  # noqa: F811
    run8(fa, Batch8([600, 40], [3000, 5000], 1, D, 128, kind="any"), 2)
    r = np.random.default_rng(2)
    run8(fa, Batch8([1] * 299 + [20], list(r.integers(20, 90, 300)), 1, D, 16), 2)


@gpu
@pytest.mark.parametrize("shared", [16, 64, 1000, 3000])
@pytest.mark.parametrize("n,Hq", [(1, 8), (3, 4), (40, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_shared_prefix(fa, shared, n, Hq, D):  # noqa: F811
    kv = [shared + x for x in (n, n + 5, n + 300, n + 64, n)]
    page = 16 if shared < 1000 else 64
    for mask in (("causal", 0, 0), ("sink_window", 400, 7)):
        run8(fa, Batch8([n, n, n, max(n - 1, 0), n], kv, 2, D, page, shared=shared, kind="any"), Hq, *mask)
