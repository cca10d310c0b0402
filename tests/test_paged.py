"""The paged cache (fa_kv_append, fa_fwd_paged) against plain float64
attention, and the refusals of its entry points.

Tolerances, derived:
  o    P is rounded to bf16 (half a step, 2^-8 of each p) before P V, so O is
       off by at most 2^-8 A with A = sum_j w_j |v_j|; the scores' own error
       (fp32 sums of exact bf16 products, ex2.approx, a soft-cap through fp32)
       stays below 4e-4 in the exponent for |s| <= 60: 4e-4 A; the bf16 output
       adds 2^-8 |O| (fp32 output: nothing); 1e-5 covers fp32 sums of O.
  lse  the same score error: 4e-4 (fp32 sums of up to a few thousand terms
       below it).
  append: products and one sum in fp32 (3 roundings of 2^-24 each on
       |x0 c| + |x1 s|), then half a bf16 step, 2^-8 |y|; copies are exact.
"""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from block_sparse_attention_fa_gb300 import synth

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
gpu = pytest.mark.gpu
FAKE = 0x10000     # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def fa():
    from block_sparse_attention_fa_gb300 import build, fa as fam
    try:
        build.build()
    except RuntimeError as e:  # no CUDA toolkit on this host
        pytest.skip(str(e))
    fam.load_library()
    return fam


# --------------------------------------------------------------- CPU: the ABI
def test_header_and_binding_agree(fa, tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fa_paged.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(fa_[a-z_]+)\s*\(", text))
    assert names == set(fa.PAGED_SYMBOLS)
    assert all(hasattr(fa.load_library(), n) for n in names)
    structs = {"fa_paged_kv": fa.PagedKVStruct, "fa_kv_append_args": fa.KVAppendArgs,
               "fa_paged_fwd_args": fa.PagedFwdArgs}
    lines = "".join(f'printf("{s} %zu\\n", sizeof({s}));' for s in structs)
    lines += "".join(f'printf("{s}.{f[0]} %zu\\n", offsetof({s}, {f[0]}));' for s, t in structs.items()
                     for f in t._fields_)
    src = tmp_path / "layout.c"
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "fa_paged.h"\nint main(void) {{ {lines} return 0; }}')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for packer, t in ((fa._PAGED_KV, fa.PagedKVStruct), (fa._KV_APPEND, fa.KVAppendArgs), (fa._MASK, fa.MaskDesc),
                      (fa._PAGED_FWD, fa.PagedFwdArgs), (fa._SCORE, fa.ScoreDesc)):
        assert packer.size == ctypes.sizeof(t)
        # the k-th value packed lands in the k-th field
        n = sum(getattr(f[1], "_length_", 1) for f in t._fields_)
        s, k = t.from_buffer_copy(packer.pack(*range(1, n + 1))), 1
        for f in t._fields_:
            got = getattr(s, f[0])
            for x in (got if hasattr(got, "__len__") else [got]):
                assert x == k, (t, f[0])
                k += 1
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        key, off = line.split()
        s, _, f = key.partition(".")
        assert int(off) == (getattr(structs[s], f).offset if f else ctypes.sizeof(structs[s])), key


def _kv(fa, **kw):
    c = fa.PagedKVStruct(2, 2, 128, 8, 16, 4, 4, FAKE, FAKE, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


CACHE_REFUSALS = [(dict(B=0), 1), (dict(Hkv=0), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1),
                  (dict(total_q=-1), 1), (dict(D=96), 2), (dict(page_size=24), 2), (dict(page_size=8), 2),
                  (dict(page_size=512), 2), (dict(page_size=0), 2), (dict(k=None), 1), (dict(v=FAKE + 8), 1),
                  (dict(page_table=None), 1), (dict(kv_len=FAKE + 2), 1), (dict(q_start=None), 1),
                  (dict(num_pages=2**31 - 1), 2), (dict(max_pages=2**31 - 1), 2)]


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS, ids=str)
def test_cache_refusals(fa, kw, status):
    lib = fa.load_library()
    c, a, f = _kv(fa, **kw), _append(fa), _fwd(fa)
    m, sc = fa.MaskDesc(), fa.ScoreDesc()
    m.kind = 1
    ws = ctypes.c_void_p(FAKE)
    assert lib.fa_kv_append(ctypes.byref(c), ctypes.byref(a), ws, None) == status
    assert lib.fa_fwd_paged(ctypes.byref(c), ctypes.byref(f), ctypes.byref(m), ctypes.byref(sc), ws, 1 << 40, ws,
                            None) == status
    assert lib.fa_paged_scratch_bytes(ctypes.byref(c), ctypes.byref(f)) == 0
    assert lib.fa_last_error()


def _append(fa, **kw):
    a = fa.KVAppendArgs()
    a.Hq, a.rot_dim, a.rope_len = 4, 64, 100
    a.q = a.k = a.v = a.q_out = a.cos = a.sin = FAKE
    a.q_stride[:] = a.q_out_stride[:] = (512, 128)
    a.k_stride[:] = a.v_stride[:] = (256, 128)
    for k, v in kw.items():
        if k.endswith("stride"):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=-1), 1), (dict(rot_dim=8), 2), (dict(rot_dim=144), 2), (dict(rot_dim=-16), 2), (dict(interleaved=2), 1),
    (dict(q=None), 1), (dict(k=FAKE + 8), 1), (dict(v=None), 1), (dict(q_out=None), 1), (dict(k_stride=(250, 128)), 1),
    (dict(q_stride=(-512, 128)), 1), (dict(q_out_stride=(64, 128), q_stride=(64, 128)), 1),
    (dict(q_out_stride=(512, 64), q_stride=(512, 64)), 1), (dict(q_stride=(1024, 128)), 1), (dict(cos=None), 1),
    (dict(sin=FAKE + 4), 1), (dict(rope_len=0), 1), (dict(positions=FAKE + 2), 1)], ids=str)
def test_append_refusals(fa, kw, status):
    lib = fa.load_library()
    c, a = _kv(fa), _append(fa, **kw)
    assert lib.fa_kv_append(ctypes.byref(c), ctypes.byref(a), ctypes.c_void_p(FAKE), None) == status
    assert lib.fa_kv_append(ctypes.byref(c), ctypes.byref(_append(fa)), None, None) == fa.ERR_INVALID_ARG
    assert lib.fa_kv_append(ctypes.byref(c), None, ctypes.c_void_p(FAKE), None) == fa.ERR_INVALID_ARG


def test_append_refuses_overlaps(fa):
    lib, ws = fa.load_library(), ctypes.c_void_p(FAKE)
    # tokens 1.. start on the heads of token 0, and heads 1.. on its tokens
    for st in ((128, 128), (256, 128), (384, 128), (128, 384), (136, 128), (504, 128)):
        a = _append(fa, q_out_stride=st, q_stride=st)
        assert lib.fa_kv_append(ctypes.byref(_kv(fa)), ctypes.byref(a), ws, None) == fa.ERR_INVALID_ARG
        assert b"overlap its rows" in lib.fa_last_error()
    # 8 pages x 2 heads x 16 tokens x 128 columns of two bytes
    for v in (FAKE, FAKE + 65536 - 16, FAKE - 65536 + 16):
        assert lib.fa_kv_append(ctypes.byref(_kv(fa, v=v)), ctypes.byref(_append(fa)), ws, None) == fa.ERR_INVALID_ARG
        assert b"k and v overlap" in lib.fa_last_error()


def _fwd(fa, **kw):
    a = fa.PagedFwdArgs()
    a.Hq, a.max_q_len = 4, 4
    a.q = a.o = a.lse = FAKE
    a.q_stride[:] = (512, 128)
    for k, v in kw.items():
        if k == "q_stride":
            a.q_stride[:] = v
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,mask,status", [
    (dict(Hq=0), {}, 1), (dict(Hq=3), {}, 1), (dict(max_q_len=0), {}, 1), (dict(shared_len=-1), {}, 1),
    (dict(shared_len=65), {}, 1), (dict(q=None), {}, 1), (dict(o=FAKE + 8), {}, 1), (dict(lse=None), {}, 1),
    (dict(q_stride=(12, 128)), {}, 1), (dict(scale=float("nan")), {}, 1), (dict(flags=2), {}, 1),
    ({}, dict(kind=3), 2), ({}, dict(kind=4), 2), ({}, dict(kind=5), 2), ({}, dict(kind=9), 2),
    ({}, dict(kind=2, window=-1), 1), ({}, dict(kind=6, window=3, prefix_len=-2), 1)], ids=str)
def test_forward_refusals(fa, kw, mask, status):
    lib = fa.load_library()
    c, a, m, sc = _kv(fa), _fwd(fa, **kw), fa.MaskDesc(), fa.ScoreDesc()
    m.kind = 1
    for k, v in mask.items():
        setattr(m, k, v)
    p = ctypes.c_void_p(FAKE)
    assert lib.fa_fwd_paged(ctypes.byref(c), ctypes.byref(a), ctypes.byref(m), ctypes.byref(sc), p, 1 << 40, p,
                            None) == status, lib.fa_last_error()


def test_forward_refusals_of_the_rest(fa):
    lib = fa.load_library()
    c, a, m, sc = _kv(fa), _fwd(fa), fa.MaskDesc(), fa.ScoreDesc()
    m.kind = 1
    p = ctypes.c_void_p(FAKE)
    call = lambda c=c, m=ctypes.byref(m), sc=ctypes.byref(sc), s=p, n=1 << 40, w=p: lib.fa_fwd_paged(  # noqa: E731
        ctypes.byref(c), ctypes.byref(a), m, sc, s, n, w, None)
    assert call(m=None) == fa.ERR_INVALID_ARG
    assert call(s=None) == fa.ERR_INVALID_ARG
    assert call(s=ctypes.c_void_p(FAKE + 8)) == fa.ERR_INVALID_ARG
    assert call(n=100) == fa.ERR_INVALID_ARG
    assert b"scratch" in lib.fa_last_error()
    assert call(w=None) == fa.ERR_INVALID_ARG
    assert call(c=_kv(fa, B=2049)) == fa.ERR_UNSUPPORTED
    assert call(c=_kv(fa, B=2048, max_pages=2**26, total_q=2**24)) == fa.ERR_UNSUPPORTED
    bad = fa.ScoreDesc()
    bad.kind, bad.softcap = 1, -1.0
    assert call(sc=ctypes.byref(bad)) == fa.ERR_INVALID_ARG
    # enough scratch for a small call is a few megabytes, and no step without rows launches anything
    assert 0 < lib.fa_paged_scratch_bytes(ctypes.byref(c), ctypes.byref(a)) < 64 << 20
    assert call(c=_kv(fa, total_q=0)) == fa.OK


# ------------------------------------------------------------------ GPU set-up
class Batch:
    """Sequences of `new` new tokens and length `kv` (new included) on shuffled pages; keys and values past kv, and
    on pages that nobody owns, are NaN; page table entries past the end are -1."""

    def __init__(self, new, kv, Hkv, D, page, seed=0, shared=0, pad=0, extra=3):
        g = np.random.default_rng(seed)
        self.new, self.kv, self.Hkv, self.D, self.page, self.shared = list(new), list(kv), Hkv, D, page, shared
        B = len(new)
        rows = [-(-n // page) for n in kv]
        first = shared // page                   # whole pages in common; the prefix's last keys are copied
        total = first + sum(max(r - first, 0) for r in rows) + extra
        ids = g.permutation(total).astype(np.int32)
        self.table = np.full((B, max(max(rows), 1) + 1), -1, np.int32)
        at = first
        for b in range(B):
            for c in range(rows[b]):
                if c < first:
                    self.table[b, c] = ids[c]
                else:
                    self.table[b, c] = ids[at]
                    at += 1
        k = synth.round_to_bf16(synth.standard_normal(seed * 2 + 1, (max(sum(kv), 1), Hkv, D)))
        v = synth.round_to_bf16(synth.standard_normal(seed * 2 + 2, (max(sum(kv), 1), Hkv, D)))
        off = np.concatenate([[0], np.cumsum(kv)])
        self.k = [k[off[b]:off[b + 1]] for b in range(B)]
        self.v = [v[off[b]:off[b + 1]] for b in range(B)]
        for b in range(1, B):
            n = min(shared, kv[b])
            self.k[b][:n], self.v[b][:n] = self.k[0][:n], self.v[0][:n]
        kc = np.full((total, Hkv, page, D), np.nan, np.float32)
        vc = kc.copy()
        for b in range(B):
            j = np.arange(kv[b])
            kc[self.table[b, j // page], :, j % page] = self.k[b]
            vc[self.table[b, j // page], :, j % page] = self.v[b]
        self.kc, self.vc = kc, vc
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.total = int(self.q_start[-1]) + pad

    def device(self):
        t = lambda x, dt: torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dt)   # noqa: E731
        return (t(self.kc, torch.bfloat16), t(self.vc, torch.bfloat16), t(self.table, torch.int32),
                t(np.array(self.kv), torch.int32), t(self.q_start, torch.int32))

    def queries(self, Hq, seed=5, scale=1.0):
        return synth.round_to_bf16(synth.standard_normal(seed, (self.total, Hq, self.D), scale))


def _score64(score, s, i, j, h, kw):
    if score == "softcap":
        return kw["softcap"] * np.tanh(s / kw["softcap"])
    if score in ("alibi", "alibi_softcap"):
        s = s - kw["slopes"][h] * np.abs(i - j)
        return s if score == "alibi" else kw["softcap"] * np.tanh(s / kw["softcap"])
    if score == "rel_bias":
        R = kw["rel_max"]
        return s + kw["rel_bias"][h][np.clip(i - j, -R, R) + R]
    return s


def reference(bt, q, mask, window, sinks, score="none", scale=None, **kw):
    """(o, lse, A) in float64, A = sum_j w_j |v_j|; rows behind the last sequence are NaN."""
    Hq = q.shape[1]
    o = np.full((bt.total, Hq, bt.D), np.nan)
    A, lse = o.copy(), np.full((bt.total, Hq), np.nan)
    scale = 1 / math.sqrt(bt.D) if scale is None else scale
    for b, (n, L) in enumerate(zip(bt.new, bt.kv)):
        i, j = np.arange(L - n, L)[:, None], np.arange(L)[None]
        see = np.ones((n, L), bool) if mask == "full" else i >= j
        if mask in ("sliding_window", "sink_window"):
            see &= (i - j <= window) | (j < (sinks if mask == "sink_window" else 0))
        for h in range(Hq):
            k, v = (x[b][:, h * bt.Hkv // Hq].astype(np.float64) for x in (bt.k, bt.v))
            rows = slice(bt.q_start[b], bt.q_start[b + 1])
            x = _score64(score, q[rows, h].astype(np.float64) @ k.T * scale, i, j, h, kw)
            x = np.where(see, x, -np.inf)
            m = x.max(-1, keepdims=True) if L else np.zeros((n, 1))
            w = np.exp(x - m)
            t = w.sum(-1, keepdims=True)
            o[rows, h], A[rows, h], lse[rows, h] = w / t @ v, w / t @ np.abs(v), (m + np.log(t))[:, 0]
    return o, lse, A


def compare(got, ref, bf16_out=True):
    (o, lse), (ro, rl, A) = got, ref
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    rows = ~np.isnan(rl)
    tol = (2.0 ** -8 + 4e-4) * A + (2.0 ** -8 * np.abs(ro) if bf16_out else 0) + 1e-5
    err = np.abs(o - ro)[rows]
    assert np.isfinite(o[rows]).all()
    assert (err <= tol[rows]).all(), f"o off by {np.nanmax(err / tol[rows]):.2f} of what it may"
    assert (np.abs(lse - rl)[rows] <= 4e-4).all(), f"lse off by {np.nanmax(np.abs(lse - rl)[rows])}"


def run(fa, bt, Hq, mask="causal", window=0, sinks=0, score="none", q_scale=1.0, out_fp32=False, shared=None, scale=None,
        max_q_len=None, **kw):
    q = bt.queries(Hq, scale=q_scale)
    dev = bt.device()
    qd = torch.from_numpy(q).cuda().to(torch.bfloat16)
    gkw = {}
    if "softcap" in kw:
        gkw["softcap"] = kw["softcap"]
    if "slopes" in kw:
        gkw["alibi_slopes"] = torch.from_numpy(kw["slopes"].astype(np.float32)).cuda()
    if "rel_bias" in kw:
        gkw.update(rel_bias=torch.from_numpy(kw["rel_bias"].astype(np.float32)).cuda().contiguous(), rel_max=kw["rel_max"])
    got = fa.fwd_paged(qd, *dev, max_q_len=max_q_len or max(max(bt.new), 1), mask=mask, window=window, sinks=sinks,
                       shared_len=bt.shared if shared is None else shared, score=score, out_fp32=out_fp32, scale=scale, **gkw)
    fa.default_workspace("cuda").check()
    compare(got, reference(bt, q, mask, window, sinks, score, scale, **kw), not out_fp32)
    return got


def score_kw(score, Hq):
    r = np.random.default_rng(3)
    return {"none": {}, "softcap": dict(softcap=5.0), "alibi": dict(slopes=r.random(Hq).astype(np.float32) * 0.3),
            "alibi_softcap": dict(slopes=r.random(Hq).astype(np.float32) * 0.3, softcap=4.0),
            "rel_bias": dict(rel_bias=r.standard_normal((Hq, 81)).astype(np.float32), rel_max=40)}[score]


SCORES = ["none", "softcap", "alibi", "alibi_softcap", "rel_bias"]
MASKS = [("full", 0, 0), ("causal", 0, 0), ("sliding_window", 70, 0), ("sink_window", 70, 5), ("sink_window", 0, 140),
         ("sliding_window", 0, 0)]


# ------------------------------------------------------------------ GPU: append
@gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 64, True), (64, 64, False), (64, 16, True),
                                               (128, 48, False), (64, 0, False), (128, 128, True)])
@pytest.mark.parametrize("fused", [True, False])
def test_append(fa, page, D, rot, interleaved, fused):
    bt = Batch([1, 0, 5, 300, 2], [1, 7, 261, 300, 130], 2, D, page, pad=3)
    kc, vc, table, kv, qs = bt.device()
    Hq, T = 6, bt.total
    x = synth.round_to_bf16(synth.standard_normal(9, (T, 10, D)))
    xd = torch.from_numpy(x).cuda().to(torch.bfloat16)
    q, k, v = (xd[:, :6], xd[:, 6:8], xd[:, 8:])
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    ang = np.random.default_rng(1).random((301, max(rot // 2, 1))) * 7
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    kw = dict(cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda()) if rot else {}
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    k0, v0 = kc.clone(), vc.clone()
    fa.kv_append(q, k, v, kc, vc, table, kv, qs, interleaved=interleaved, q_out=out, **kw)
    fa.default_workspace("cuda").check()

    def turned(a, i):
        a = a.astype(np.float64)
        y, mag = a.copy(), np.zeros_like(a)
        if rot:
            p0 = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
            p1 = p0 + 1 if interleaved else p0 + rot // 2
            c, s = cos[i].astype(np.float64), sin[i].astype(np.float64)
            y[..., p0], y[..., p1] = a[..., p0] * c - a[..., p1] * s, a[..., p0] * s + a[..., p1] * c
            mag[..., p0], mag[..., p1] = np.abs(a[..., p0] * c) + np.abs(a[..., p1] * s), \
                np.abs(a[..., p0] * s) + np.abs(a[..., p1] * c)
        return y, np.where(mag > 0, 2.0 ** -8 * np.abs(y) + 3 * 2.0 ** -24 * mag, 0)

    want_k, want_v = k0.double().cpu().numpy(), v0.double().cpu().numpy()
    tol_k = np.zeros_like(want_k)
    got_q = out.double().cpu().numpy()
    for b, (n, L) in enumerate(zip(bt.new, bt.kv)):
        for t in range(n):
            i, r = L - n + t, bt.q_start[b] + t
            y, tol = turned(x[r, :6], i)
            assert (np.abs(got_q[r] - y) <= tol).all()
            pg, sl = bt.table[b, i // page], i % page
            want_k[pg, :, sl], tol_k[pg, :, sl] = turned(x[r, 6:8], i)
            want_v[pg, :, sl] = x[r, 8:]
    assert (got_q[bt.q_start[-1]:] == 7).all()                 # rows behind the last sequence
    got_k, got_v = kc.double().cpu().numpy(), vc.double().cpu().numpy()
    nan = np.isnan(want_k)
    assert np.array_equal(nan, np.isnan(got_k)) and (np.abs(got_k - want_k)[~nan] <= tol_k[~nan]).all()
    assert np.array_equal(got_v, want_v, equal_nan=True)


@gpu
def test_append_in_place_and_positions(fa):
    bt = Batch([3, 2], [20, 40], 2, 64, 16)
    dev = bt.device()
    x = torch.randn(5, 8, 64, device="cuda").to(torch.bfloat16)
    ang = torch.rand(50, 32, device="cuda")
    pos = torch.tensor([4, 0, 49, 7, 7], dtype=torch.int32, device="cuda")
    kw = dict(cos=ang.cos(), sin=ang.sin(), positions=pos)
    q = x[:, :4].contiguous()
    apart = fa.kv_append(q.clone(), x[:, 4:6], x[:, 6:], *dev, **kw)
    same = fa.kv_append(q, x[:, 4:6], x[:, 6:], *dev, q_out=q, **kw)
    assert same is q and torch.equal(apart, q)
    # positions name the tables' rows, not the slots
    c, s = ang.cos()[pos.long()][:, None], ang.sin()[pos.long()][:, None]
    a, b = x[:, :4, :32].float(), x[:, :4, 32:].float()
    want = torch.cat([a * c - b * s, a * s + b * c], -1)
    assert ((q.float() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all()
    kc, vc, table = dev[0], dev[1], bt.table
    assert torch.equal(vc[table[1, 39 // 16], :, 39 % 16], x[4, 6:])
    assert fa.kv_append(None, x[:, 4:6], x[:, 6:], *dev) is None      # no queries, no rotation
    assert torch.equal(kc[table[0, 17 // 16], :, 17 % 16], x[0, 4:6])
    fa.default_workspace("cuda").check()


# ------------------------------------------------------------ GPU: single tokens
@gpu
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mask,window,sinks", MASKS)
def test_decode_masks(fa, page, D, mask, window, sinks):
    run(fa, Batch([1, 1, 1, 1, 1], [1, 700, 129, 128, 300], 2, D, page), 8, mask, window, sinks)


@gpu
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("out_fp32", [False, True])
def test_decode_scores(fa, score, D, out_fp32):
    run(fa, Batch([2, 1, 0, 3], [500, 40, 10, 333], 2, D, 16), 6, "sink_window", 200, 3, score=score, out_fp32=out_fp32,
        **score_kw(score, 6))


@gpu
@pytest.mark.parametrize("Hq,Hkv,n", [(1, 1, 1), (1, 1, 16), (16, 1, 1), (4, 4, 3), (9, 3, 5), (14, 2, 2), (5, 1, 3)])
def test_decode_groups(fa, Hq, Hkv, n):
    run(fa, Batch([n, 1, n], [n, 150, 400], Hkv, 128, 32), Hq)


@gpu
@pytest.mark.parametrize("kv", [[1], [2], [127], [128], [129], [5000], [40000], [3] * 70, [1, 30000, 1, 1], [257] * 300])
def test_decode_lengths(fa, kv):
    run(fa, Batch([1] * len(kv), kv, 2, 64, 16), 4)


@gpu
def test_decode_largest_batch(fa):
    run(fa, Batch([1] * 2048, [(i * 37) % 50 + 1 for i in range(2048)], 1, 64, 16), 2)


@gpu
@pytest.mark.parametrize("B", [1000, 1001, 1999, 2001])
@pytest.mark.parametrize("lengths", ["short", "mixed"])
def test_decode_many_sequences(fa, B, lengths):
    new = [0 if b % 5 == 3 or 300 < b < 340 else 1 for b in range(B)]
    kv = [(b * 37) % 50 + 1 + (900 if lengths == "mixed" and b % 97 == 5 else 0) for b in range(B)]
    run(fa, Batch(new, kv, 2, 64, 16), 4)


@gpu
@pytest.mark.parametrize("Hq,shared", [(17, 0), (2, 16), (17, 16)])
def test_largest_batch_of_the_other_kernels(fa, Hq, shared):
    run(fa, Batch([1] * 2048, [shared + (i * 37) % 50 + 1 for i in range(2048)], 1, 64, 16, shared=shared), Hq)


# ------------------------------------------------------------- GPU: many rows
@gpu
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mask,window,sinks", MASKS)
def test_chunk_masks(fa, page, D, mask, window, sinks):
    run(fa, Batch([100, 1, 37, 0, 260], [100, 300, 500, 20, 261], 2, D, page), 6, mask, window, sinks)


@gpu
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("out_fp32", [False, True])
def test_chunk_scores(fa, score, D, out_fp32):
    run(fa, Batch([70, 20, 1], [300, 40, 333], 2, D, 32), 4, "sink_window", 100, 3, score=score, out_fp32=out_fp32,
        **score_kw(score, 4))


@gpu
@pytest.mark.parametrize("Hq,Hkv,n", [(1, 1, 17), (1, 1, 257), (3, 1, 100), (32, 1, 30), (5, 5, 129), (7, 1, 40), (300, 1, 2)])
def test_chunk_groups(fa, Hq, Hkv, n):
    run(fa, Batch([n, 2], [n + 5, 150], Hkv, 64, 16), Hq)


@gpu
@pytest.mark.parametrize("new,kv", [([600], [600]), ([513, 1, 900], [2000, 3000, 900]), ([128] * 9, [128 + 64 * i for i in range(9)])])
def test_chunk_lengths(fa, new, kv):
    run(fa, Batch(new, kv, 2, 128, 64), 8)


@gpu
@pytest.mark.parametrize("new,kv", [([1] * 48, [3] * 24 + [2500] * 24), ([1] * 300, [64 + (b % 7) for b in range(300)]),
                                    ([2, 1, 2] * 30, [5, 1, 900] * 30)])
def test_decode_short_beside_long(fa, new, kv):
    run(fa, Batch(new, kv, 4, 64, 32), 8)


@gpu
@pytest.mark.parametrize("new,kv,Hq,Hkv", [([2100], [2100], 4, 1), ([700] * 3, [700] * 3, 8, 2), ([130] * 15, [130] * 15, 4, 2),
                                           ([17, 1, 300, 40] * 5, [17, 2000, 300, 3000] * 5, 4, 1)])
def test_prompts(fa, new, kv, Hq, Hkv):
    run(fa, Batch(new, kv, Hkv, 64, 64), Hq)


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,Hq", [(1, 24), (4, 8), (9, 8)])
def test_few_rows_in_many_parts(fa, n, Hq, D):
    run(fa, Batch([n], [40000], 1, D, 16), Hq)


@gpu
@pytest.mark.parametrize("q_scale", [0.1, 1.0, 8.0, 60.0])
@pytest.mark.parametrize("cap", [2.0, 50.0])
@pytest.mark.parametrize("n", [1, 40])
def test_softcap_ranges(fa, n, cap, q_scale):
    run(fa, Batch([n] * 3, [n + 300, n + 90, n + 1000], 2, 64, 32), 8, score="softcap", softcap=cap, q_scale=q_scale)


@gpu
def test_large_scores_rescale(fa):
    """Scores that grow along the keys: the running max rises again and again."""
    for new in ([1], [80]):
        bt = Batch(new, [900], 1, 64, 16)
        ramp = np.linspace(0.1, 3.0, 900, dtype=np.float32)[:, None, None]
        bt.k[0][:] = synth.round_to_bf16(np.abs(bt.k[0]) * ramp)
        j = np.arange(900)
        bt.kc[bt.table[0, j // 16], :, j % 16] = bt.k[0]
        q = np.abs(bt.queries(2))
        bt.queries = lambda Hq, scale=1.0, q=q: q
        run(fa, bt, 2, scale=0.2)
        run(fa, bt, 2, scale=0.2, out_fp32=True)


# ---------------------------------------------------------- GPU: shared prefix
@gpu
@pytest.mark.parametrize("shared", [16, 128, 200, 1000])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mask,window,sinks", MASKS)
def test_shared_masks(fa, shared, D, mask, window, sinks):
    run(fa, Batch([1, 4, 2, 1], [shared + x for x in [3, 300, 30, 130]], 2, D, 16, shared=shared), 6, mask, window, sinks)


@gpu
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("n", [1, 50])
def test_shared_scores(fa, score, n):
    run(fa, Batch([n, 1, n], [700 + n, 620, 601 + n], 2, 128, 64, shared=600), 6, score=score, **score_kw(score, 6))


@gpu
@pytest.mark.parametrize("B,n,Hq,Hkv", [(70, 1, 8, 2), (3, 100, 4, 1), (1, 1, 4, 4), (130, 3, 5, 1), (2, 300, 8, 2)])
@pytest.mark.parametrize("out_fp32", [False, True])
def test_shared_sizes(fa, B, n, Hq, Hkv, out_fp32):
    new = [max(1, n - 7 * (b % 3)) for b in range(B)]
    run(fa, Batch(new, [333 + m + 29 * (b % 5) for b, m in enumerate(new)], Hkv, 64, 32, shared=333), Hq, out_fp32=out_fp32)


@gpu
def test_shared_all_of_it_and_rows_without_tokens(fa):
    """Queries inside the prefix (nothing of their own behind it), and a sequence without new tokens."""
    run(fa, Batch([5, 0, 5], [200, 300, 200], 2, 64, 16, shared=200), 4)
    run(fa, Batch([5, 0, 5], [200, 3, 260], 2, 64, 16, shared=196), 4)


@gpu
def test_shared_equals_separate(fa):
    bt = Batch([2] * 9, [500 + 40 * b for b in range(9)], 2, 128, 16, shared=480)
    a, b = run(fa, bt, 8, shared=480), run(fa, bt, 8, shared=0)
    assert torch.allclose(a[1], b[1], atol=1e-5)
    assert (a[0].float() - b[0].float()).abs().max() < 0.05


# ------------------------------------------------- GPU: what can go wrong beside
@gpu
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("shared", [0, 64])
def test_padding_rows_are_left(fa, n, shared):
    bt = Batch([n, n], [90 + n, 300], 2, 64, 16, shared=shared, pad=5)
    dev, q = bt.device(), torch.from_numpy(bt.queries(4)).cuda().to(torch.bfloat16)
    q[bt.q_start[-1]:] = float("nan")
    out = torch.full((bt.total, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((bt.total, 4), 3.0, device="cuda")
    fa.fwd_paged(q, *dev, max_q_len=n, shared_len=shared, out=out, lse=lse)
    fa.default_workspace("cuda").check()
    compare((out, lse), reference(bt, bt.queries(4), "causal", 0, 0))
    assert (out[bt.q_start[-1]:] == 3).all() and (lse[bt.q_start[-1]:] == 3).all()


@gpu
@pytest.mark.parametrize("n", [1, 40])
def test_strided_queries(fa, n):
    bt = Batch([n, n], [90 + n, 300], 2, 64, 16)
    dev, q = bt.device(), bt.queries(4)
    wide = torch.zeros((bt.total, 8, 72), dtype=torch.bfloat16, device="cuda")
    wide[:, ::2, :64] = torch.from_numpy(q).cuda().to(torch.bfloat16)
    got = fa.fwd_paged(wide[:, ::2, :64], *dev, max_q_len=n)
    fa.default_workspace("cuda").check()
    compare(got, reference(bt, q, "causal", 0, 0))


@gpu
@pytest.mark.parametrize("n", [2, 40])
def test_freed_pages_are_not_read(fa, n):
    """Pages before the window go back to the pool: their table entries name nothing."""
    bt = Batch([n], [1000], 2, 64, 16)
    dev = bt.device()
    q = bt.queries(4)
    first = (1000 - n - 100) // 16
    dev[2][0, 1:first] = -1                     # the sinks' page stays
    kept = torch.from_numpy(bt.table[0, [0] + list(range(first, 63))]).long()
    keep = torch.zeros(dev[0].shape[0], dtype=torch.bool)
    keep[kept] = True
    dev[0][~keep.cuda()] = float("nan")
    dev[1][~keep.cuda()] = float("nan")
    got = fa.fwd_paged(torch.from_numpy(q).cuda().to(torch.bfloat16), *dev, max_q_len=n, mask="sink_window", window=100,
                       sinks=4)
    fa.default_workspace("cuda").check()
    compare(got, reference(bt, q, "sink_window", 100, 4))


@gpu
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("shared", [0, 32])
@pytest.mark.parametrize("fault", ["page", "page_high", "kv_long", "kv_short", "q_order", "q_past", "n_long", "negative"])
def test_bad_numbers_are_reported(fa, n, shared, fault):
    """Every one of them ends in a check of the kernels, never in an access outside the arrays: tests/test_paged_units.py
    compares those checks with the definition on the CPU.  The other sequences are not affected."""
    bt = Batch([n, n, n], [100 + n, 200 + n, 300], 2, 64, 16, shared=shared)
    kc, vc, table, kv, qs = bt.device()
    q = bt.queries(4)
    qd = torch.from_numpy(q).cuda().to(torch.bfloat16)
    max_q = n
    good = [0, 2]
    if fault == "page":
        table[1, 9] = -1
    elif fault == "page_high":
        table[1, 9] = kc.shape[0]
    elif fault == "kv_long":
        kv[1] = table.shape[1] * 16 + 1
    elif fault == "kv_short":
        kv[1] = n - 1
    elif fault == "q_order":
        qs[1], good = 2 * n + 1, []            # a q_start that decreases leaves every row undefined
    elif fault == "q_past":
        qs[3], good = 3 * n + 1, [0, 1]
    elif fault == "n_long":
        max_q, good = max(n - 1, 1), []
        if n == 1:
            qs[:] = torch.tensor([0, 2, 2, 3], dtype=torch.int32)
    else:
        kv[1] = -5
    out = torch.zeros((bt.total, 4, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((bt.total, 4), device="cuda")
    fa.fwd_paged(qd, kc, vc, table, kv, qs, max_q_len=max_q, shared_len=shared, out=out, lse=lse)
    with pytest.raises(fa.FAError) as e:
        fa.default_workspace("cuda").check()
    assert e.value.status == fa.ERR_DEVICE_CHECK and "sequence" in str(e.value)
    fa.default_workspace("cuda").check()        # cleared
    ro, rl, A = reference(bt, q, "causal", 0, 0)
    for b in range(3):
        if b not in good:
            ro[bt.q_start[b]:bt.q_start[b + 1]] = rl[bt.q_start[b]:bt.q_start[b + 1]] = np.nan
    if good:
        compare((out, lse), (ro, rl, A))


@gpu
@pytest.mark.parametrize("fault", ["page", "kv_long", "q_order", "rope"])
def test_append_reports_bad_numbers(fa, fault):
    bt = Batch([2, 2, 2], [20, 30, 40], 1, 64, 16)
    kc, vc, table, kv, qs = bt.device()
    x = torch.randn(6, 3, 64, device="cuda").to(torch.bfloat16)
    cos = torch.ones(29 if fault == "rope" else 64, 32, device="cuda")
    if fault == "page":
        table[1, 1] = 1 << 20
    elif fault == "kv_long":
        kv[1] = 10000
    elif fault == "q_order":
        qs[1] = 5
    k0 = kc.clone()
    fa.kv_append(x[:, :1], x[:, 1:2], x[:, 2:], kc, vc, table, kv, qs, cos=cos, sin=cos * 0)
    with pytest.raises(fa.FAError) as e:
        fa.default_workspace("cuda").check()
    assert e.value.status == fa.ERR_DEVICE_CHECK
    if fault != "q_order":
        assert torch.equal(vc[bt.table[0, 1], :, 19 % 16], x[1, 2:]) and torch.equal(vc[bt.table[2, 2], :, 7], x[5, 2:]) \
            == (fault != "rope")
        changed = (kc != k0) & ~(torch.isnan(kc) & torch.isnan(k0))
        assert not changed[bt.table[1, 1], :, 13].any()          # position 29 of sequence 1


@gpu
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("shared", [0, 64])
def test_time_limit_changes_nothing(fa, n, shared):
    """A call whose waits do not run out reports nothing, and its results do not depend on the limit."""
    bt = Batch([n, n], [90 + n, 300], 2, 64, 16, shared=shared)
    dev, q = bt.device(), torch.from_numpy(bt.queries(4)).cuda().to(torch.bfloat16)
    a = fa.fwd_paged(q, *dev, max_q_len=n, shared_len=shared, timeout_ms=5000)
    b = fa.fwd_paged(q, *dev, max_q_len=n, shared_len=shared)
    fa.default_workspace("cuda").check()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------- GPU: used together
@gpu
@pytest.mark.parametrize("shared", [0, 48])
def test_serving_loop(fa, shared):
    """A prompt chunk, then single tokens: each step appends and attends, in one captured graph per kind of step that
    follows the lengths on the device.  Against float64 attention over what was appended."""
    Hq, Hkv, D, page, B = 6, 2, 64, 16, 3
    bt = Batch([30, 41, 55], [shared + 30, shared + 41, shared + 55], Hkv, D, page, shared=shared)
    grown = np.full((B, bt.table.shape[1] + 3), -1, np.int32)
    spare = 0
    kc, vc, _, kv, qs = bt.device()
    kc = torch.cat([kc, torch.full((12, *kc.shape[1:]), float("nan"), dtype=kc.dtype, device="cuda")])
    vc = torch.cat([vc, torch.full((12, *vc.shape[1:]), float("nan"), dtype=vc.dtype, device="cuda")])
    for b in range(B):
        own = [x for x in bt.table[b] if x >= 0]
        grown[b, :len(own)] = own
        for c in range(len(own), (bt.kv[b] + 4) // page + 1):
            grown[b, c] = len(bt.kc) + spare
            spare += 1
    table = torch.from_numpy(grown).cuda()
    ang = np.random.default_rng(2).random((400, D // 2)) * 6
    cos, sin = torch.from_numpy(np.cos(ang)).cuda().float(), torch.from_numpy(np.sin(ang)).cuda().float()
    keys = [bt.k[b][:shared].astype(np.float64) for b in range(B)]
    vals = [bt.v[b][:shared].astype(np.float64) for b in range(B)]

    def turn(x, i):
        x = torch.from_numpy(x).float()
        c, s = cos.cpu()[i][:, None], sin.cpu()[i][:, None]
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1).to(torch.bfloat16)

    def step(x):
        q = fa.kv_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, table, kv, qs, cos=cos, sin=sin)
        return q, fa.fwd_paged(q, kc, vc, table, kv, qs, max_q_len=int(x.shape[0]) if x.shape[0] > B else 1,
                               shared_len=shared)

    def check(x, q, got, new, lens):
        ro = np.zeros(got[0].shape)
        rl, A = np.zeros(got[1].shape), np.zeros(got[0].shape)
        x, r = x.double().cpu().numpy(), 0
        qq = q.double().cpu().numpy()
        for b in range(B):
            i = np.arange(lens[b] - new[b], lens[b])
            keys[b] = np.concatenate([keys[b], turn(x[r:r + new[b], Hq:Hq + Hkv], i).double().numpy()])
            vals[b] = np.concatenate([vals[b], x[r:r + new[b], Hq + Hkv:]])
            for h in range(Hq):
                g = h * Hkv // Hq
                s = qq[r:r + new[b], h] @ keys[b][:, g].T / math.sqrt(D)
                s = np.where(i[:, None] >= np.arange(lens[b])[None], s, -np.inf)
                m = s.max(-1, keepdims=True)
                w = np.exp(s - m)
                t = w.sum(-1, keepdims=True)
                ro[r:r + new[b], h], A[r:r + new[b], h] = w / t @ vals[b][:, g], w / t @ np.abs(vals[b][:, g])
                rl[r:r + new[b], h] = (m + np.log(t))[:, 0]
            r += new[b]
        # a rotated key may round to the neighbour of the one made here (fused products): half a bf16 step of k and
        # of q moves a score by up to 2^-8 |s| terms
        o, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
        assert (np.abs(o - ro) <= (2.0 ** -8 + 0.02) * A + 2.0 ** -8 * np.abs(ro) + 1e-5).all()
        assert (np.abs(lse - rl) <= 0.02).all()

    x = torch.randn(126, Hq + 2 * Hkv, D, device="cuda").to(torch.bfloat16)
    q, got = step(x)
    check(x, q, got, bt.new, bt.kv)
    qs.copy_(torch.arange(B + 1, dtype=torch.int32))
    lens = list(bt.kv)
    x1 = torch.randn(B, Hq + 2 * Hkv, D, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv += 1
        lens = [n + 1 for n in lens]
        q, got = step(x1)
    torch.cuda.current_stream().wait_stream(side)
    check(x1, q, got, [1] * B, lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, got = step(x1)
    for _ in range(3):
        x1.copy_(torch.randn(B, Hq + 2 * Hkv, D, device="cuda"))
        kv += 1
        lens = [n + 1 for n in lens]
        graph.replay()
        check(x1, q, got, [1] * B, lens)
    fa.default_workspace("cuda").check()


@gpu
@pytest.mark.parametrize("n", [1, 40])
def test_two_graphs_at_once(fa, n):
    """Two captured calls replayed on two streams together: each has its own scratch."""
    a = Batch([n] * 5, [800 + 100 * b for b in range(5)], 2, 64, 16, seed=1, shared=0)
    b = Batch([n] * 7, [1200 - 90 * b for b in range(7)], 2, 64, 16, seed=2, shared=320)
    calls = []
    for bt in (a, b):
        dev, q = bt.device(), torch.from_numpy(bt.queries(4)).cuda().to(torch.bfloat16)
        fa.fwd_paged(q, *dev, max_q_len=n, shared_len=bt.shared)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = fa.fwd_paged(q, *dev, max_q_len=n, shared_len=bt.shared)
        calls.append((bt, g, got, dev, q))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s1):
            calls[0][1].replay()
        with torch.cuda.stream(s2):
            calls[1][1].replay()
    torch.cuda.synchronize()
    for bt, _, got, _, _ in calls:
        compare(got, reference(bt, bt.queries(4), "causal", 0, 0))


@gpu
def test_other_stream_and_repeatability(fa):
    bt = Batch([1] * 6, [100 + 700 * b for b in range(6)], 2, 128, 64)
    dev, q = bt.device(), torch.from_numpy(bt.queries(8)).cuda().to(torch.bfloat16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    first = fa.fwd_paged(q, *dev, max_q_len=1, stream=s)
    s.synchronize()
    for _ in range(20):
        again = fa.fwd_paged(q, *dev, max_q_len=1)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    compare(first, reference(bt, bt.queries(8), "causal", 0, 0))


@gpu
def test_outputs_on_another_stream_are_its_own(fa):
    """What a call on another stream allocates is not memory that the current stream has just given back, and may
    still be writing."""
    bt = Batch([3] * 5, [40 + 9 * b for b in range(5)], 2, 64, 16)
    kc, vc, table, kv, qs = bt.device()
    q = torch.from_numpy(bt.queries(4)).cuda().to(torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for call in (lambda: fa.fwd_paged(q, kc, vc, table, kv, qs, max_q_len=3, stream=s),
                 lambda: (fa.kv_append(q, q[:, :2], q[:, 2:], kc.clone(), vc.clone(), table, kv, qs, stream=s),)):
        like = [torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")]
        freed = {t.data_ptr() for t in like}
        del like
        s.wait_stream(torch.cuda.current_stream())
        got = call()
        assert not freed & {t.data_ptr() for t in got}
        torch.cuda.current_stream().wait_stream(s)
    want = fa.fwd_paged(q, kc, vc, table, kv, qs, max_q_len=3)
    got = fa.fwd_paged(q, kc, vc, table, kv, qs, max_q_len=3, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
def test_append_head_major_output(fa):
    """q_out's tokens may lie within the head stride."""
    bt = Batch([70, 3], [80, 3], 2, 64, 16)
    kc, vc, table, kv, qs = bt.device()
    q = torch.from_numpy(bt.queries(4)).cuda().to(torch.bfloat16)
    angle = torch.rand(100, 32, device="cuda")
    kw = dict(cos=angle.cos(), sin=angle.sin())
    want = fa.kv_append(q, q[:, :2], q[:, 2:], kc, vc, table, kv, qs, **kw)
    out = torch.zeros(4, q.shape[0], 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    fa.kv_append(q, q[:, :2], q[:, 2:], kc, vc, table, kv, qs, q_out=out, **kw)
    assert torch.equal(out, want)


@gpu
@pytest.mark.parametrize("n", [1, 40])
def test_pages_past_32_bits(fa, n):
    """A cache whose last pages lie 2^33 bytes (2^32 elements) behind its first: the same step on the same pages in
    a small cache gives the same bits."""
    page, Hkv, D, far = 256, 8, 128, 16384 + 8
    bt = Batch([n, n], [900, 2000], Hkv, D, page)
    kc, vc, table, kv, qs = bt.device()
    ids = torch.linspace(0, far - 1, kc.shape[0], device="cuda").round().long().flip(0)
    big = [torch.empty((far, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for x, y in zip(big, (kc, vc)):
        x[ids] = y
    there = torch.where(table >= 0, ids[table.clamp(min=0).long()], table.long()).to(torch.int32)
    q = torch.from_numpy(bt.queries(32)).cuda().to(torch.bfloat16)
    for step in range(2):
        want = fa.fwd_paged(q, kc, vc, table, kv, qs, max_q_len=n)
        got = fa.fwd_paged(q, *big, there, kv, qs, max_q_len=n)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        if step == 0:
            rows = q.flip(0)
            for k, v, t in ((kc, vc, table), (*big, there)):
                fa.kv_append(None, rows[:, :Hkv], rows[:, Hkv:2 * Hkv], k, v, t, kv, qs)
    assert torch.equal(big[0][ids].view(torch.int16), kc.view(torch.int16))
    fa.default_workspace("cuda").check()


@gpu
def test_binding_refusals(fa):
    bt = Batch([1, 1], [20, 30], 2, 64, 16)
    kc, vc, table, kv, qs = bt.device()
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    good = (kc, vc, table, kv, qs)
    for args, kw in [((q.float(), *good), {}), ((q[:, :, :32], *good), {}), ((q.transpose(0, 2), *good), {}),
                     ((q, kc.float(), vc, table, kv, qs), {}), ((q, kc[:, :1], vc, table, kv, qs), {}),
                     ((q, kc, vc, table.long(), kv, qs), {}), ((q, kc, vc, table, kv[:1], qs), {}),
                     ((q, kc, vc, table, kv, qs[:2]), {}), ((q, kc, vc, table.cpu(), kv, qs), {}),
                     ((q, *good), dict(out=q[:1])), ((q, *good), dict(lse=torch.zeros(2, 3, device="cuda"))),
                     ((q, *good), dict(score="alibi", alibi_slopes=torch.zeros(2, device="cuda"))),
                     ((q, *good), dict(mask="causal", sinks=2)), ((q, *good), dict(mask="nothing"))]:
        with pytest.raises(ValueError):
            fa.fwd_paged(*args, **kw)
    with pytest.raises(fa.FAError):
        fa.fwd_paged(q, *good, mask="document")
    with pytest.raises(fa.FAError):
        fa.fwd_paged(q, *good, scratch=torch.zeros(64, device="cuda"))
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    for args, kw in [((q, k[:1], k, *good), {}), ((q, k, k.float(), *good), {}), ((q[:1], k, k, *good), {}),
                     ((q, k, k, *good), dict(cos=torch.zeros(5, 16, device="cuda"))),
                     ((q, k, k, *good), dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda"))),
                     ((q, k, k, *good), dict(q_out=q[:, :2]))]:
        with pytest.raises(ValueError):
            fa.kv_append(*args, **kw)
    # no rows at all
    empty = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    o, lse = fa.fwd_paged(empty, kc, vc, table, kv, zero)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    fa.kv_append(empty, empty[:, :2], empty[:, :2], kc, vc, table, kv, zero)
    fa.default_workspace("cuda").check()


@gpu
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("shared", [0, 64])
def test_after_other_work_in_a_graph(fa, n, shared):
    """A captured call behind a copy, a fill, a library kernel and another paged call: its kernels start early, but
    read nothing before what comes in front is done."""
    bt = Batch([n, n, n], [400 + n, 90 + n, 300 + n], 2, 64, 16, shared=shared)
    dev = bt.device()
    q = torch.from_numpy(bt.queries(4)).cuda().to(torch.bfloat16)
    src, qd, kv = q.clone(), torch.zeros_like(q), torch.zeros_like(dev[3])
    args = (dev[0], dev[1], dev[2], kv, dev[4])
    call = lambda: fa.fwd_paged(qd, *args, max_q_len=n, shared_len=shared)   # noqa: E731
    kv.copy_(dev[3])
    qd.copy_(src)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qd.zero_()
        kv.zero_()
        torch.cuda._sleep(200000)
        kv.add_(dev[3])
        qd.copy_(src)
        first = call()
        qd.copy_(first[0])
        qd.copy_(src)
        second = call()
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    ref = reference(bt, bt.queries(4), "causal", 0, 0)
    compare(first, ref)
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])


@gpu
def test_threads_on_one_stream(fa):
    """Calls of several threads on one stream share the binding's scratch: each call's launches stay together."""
    import threading
    bts = [Batch([1] * 4, [300 + 900 * k + 50 * b for b in range(4)], 2, 64, 16, seed=k) for k in range(4)]
    work = [(bt, bt.device(), torch.from_numpy(bt.queries(4)).cuda().to(torch.bfloat16)) for bt in bts]
    torch.cuda.synchronize()
    got = [[] for _ in bts]

    def loop(k):
        for _ in range(30):
            got[k].append(fa.fwd_paged(work[k][2], *work[k][1], max_q_len=1))
    ts = [threading.Thread(target=loop, args=(k,)) for k in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    for k, bt in enumerate(bts):
        ref = reference(bt, bt.queries(4), "causal", 0, 0)
        for x in got[k]:
            compare(x, ref)
