"""fa_paged_step beside its neighbours: appends that follow at once, arrays that are the same."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_paged import FAKE, fa  # noqa: F401  (fa: the fixture)
from tests.test_paged_step import Server, _args, mixed, same, step

gpu = pytest.mark.gpu


# ---------------------------------------------------------------- appends behind it
@gpu
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("how", ["eager", "captured"])
def test_an_append_behind_a_step_of_many_rows(fa, bits, how):  # noqa: F811
    """Steps of several CTAs, each with its append directly behind it: every token where the step put it."""
    page, B, Hkv, D = 16, 40, 2, 64
    s = [Server(*mixed(B, page, k, 700, 900), page, spare=50, seed=k) for k in range(6)]
    total, width, pages = (max(f(x) for x in s) for f in (lambda x: x.total, lambda x: x.table.shape[1], lambda x: x.free.size))
    assert total > 2 * 2048                      # three CTAs of the step, or more
    for x in s:
        x.total = total
        x.table = np.pad(x.table, ((0, 0), (0, width - x.table.shape[1])), constant_values=-1)
        x.free = np.pad(x.free, (0, pages - x.free.size), constant_values=-7)
    d = s[0].device()
    r = torch.Generator().manual_seed(1)
    # whole numbers up to 8, which e4m3 holds, and in each row one of 8, so that no scale is larger in one page than in another
    rows = torch.randint(-8, 9, (total, 2 * Hkv, D), generator=r)
    rows[:, :, 5] = 8
    rows = rows.cuda().to(torch.bfloat16)
    dtype = torch.bfloat16 if bits == 16 else torch.float8_e4m3fn
    cache = [torch.zeros((pages, Hkv, page, D), device="cuda").to(dtype) for _ in range(2)]
    scales = dict(k_scale=torch.zeros((pages, Hkv), device="cuda"), v_scale=torch.zeros((pages, Hkv), device="cuda")) \
        if bits == 8 else {}
    cos, sin = torch.ones((2000, D // 2), device="cuda"), torch.zeros((2000, D // 2), device="cuda")

    def both():
        got = step(fa, s[0], d)
        fa.kv_append(None, rows[:, :Hkv], rows[:, Hkv:], *cache, d["table"], d["kv"], got[0], **scales, cos=cos, sin=sin,
                     positions=got[2])
        return got

    both()
    torch.cuda.synchronize()
    if how == "captured":
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = both()
    for x in s + s:
        for k, v in x.device().items():
            d[k].copy_(v)
        for z in (*cache, *scales.values()):
            z.zero_()
        if how == "captured":
            g.replay()
        else:
            got = both()
        want = x.want()
        same(d, got, want)
        slots = want[5][:int(x.new.sum())]
        for z, part, name in zip(cache, (rows[:, :Hkv], rows[:, Hkv:]), ("k_scale", "v_scale")):
            values = z.float()
            if bits == 8:
                values = values * scales[name][:, :, None, None]
            values = values.permute(0, 2, 1, 3).reshape(pages * page, Hkv, D).cpu()
            assert torch.equal(values[slots], part[:len(slots)].float().cpu())
            other = np.ones(pages * page, bool)
            other[slots] = False
            assert not values[other].any()
    fa.default_workspace("cuda").check()


@gpu
@pytest.mark.parametrize("bits", [16, 8])
def test_an_append_of_what_the_one_before_it_rotated(fa, bits):  # noqa: F811
    """q_out of one append as k of the next, directly behind it: as with a wait between them."""
    page, B, H, D, n = 16, 300, 4, 128, 20
    dtype = torch.bfloat16 if bits == 16 else torch.float8_e4m3fn
    x = torch.randn((B * n, H, D), device="cuda").to(torch.bfloat16)
    table = torch.arange(2 * B, dtype=torch.int32, device="cuda").view(B, 2)
    kv = torch.full((B,), n, dtype=torch.int32, device="cuda")
    starts = n * torch.arange(B + 1, dtype=torch.int32, device="cuda")
    ang = torch.rand((32, D // 2), device="cuda")
    got = []
    for wait in (True, False, False, False):
        cache = [torch.zeros((2 * B, H, page, D), device="cuda").to(dtype) for _ in range(2)]
        more = dict(k_scale=torch.zeros((2 * B, H), device="cuda"), v_scale=torch.zeros((2 * B, H), device="cuda")) \
            if bits == 8 else {}
        other = [c.clone() for c in cache], {k: v.clone() for k, v in more.items()}
        out = torch.zeros_like(x)
        torch.cuda.synchronize()
        fa.kv_append(x, x, x, *other[0], table, kv, starts, **other[1], cos=ang.cos(), sin=ang.sin(), q_out=out)
        if wait:
            torch.cuda.synchronize()
        fa.kv_append(None, out, out, *cache, table, kv, starts, **more)
        got.append([t.clone().view(torch.uint8) for t in (*cache, *more.values())])
    fa.default_workspace("cuda").check()
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


# ------------------------------------------------------------- keep_len as an output
def test_keep_len_is_no_output(fa):  # noqa: F811
    """A step that cannot be made writes kv_len to kv_len_out: that must not be what it kept."""
    lib, a = fa.load_library(), _args(fa)
    for kw in (dict(kv_len_out=a.keep_len), dict(kv_len_out=a.keep_len + 4), dict(kv_len_out=a.kv_len, keep_len=a.kv_len + 8)):
        assert lib.fa_paged_step(ctypes.byref(_args(fa, **kw)), FAKE, None) == fa.ERR_INVALID_ARG
        assert b"kv_len_out and keep_len overlap" in lib.fa_last_error()


@gpu
@pytest.mark.parametrize("pad", [0, 6000])
def test_keep_len_may_be_kv_len(fa, pad):  # noqa: F811
    """All tokens kept, said by the same array; in place or not; and where the step cannot be made."""
    old = [32, 50, 9, 0]
    for place in (True, False):
        s = Server(old, old, [1, 70, 2, 33], 16, pad=pad)
        d = s.device()
        d["keep"] = d["kv"]
        out = d["kv"] if place else torch.empty_like(d["kv"])
        same(d, step(fa, s, d, kv_len_out=out), s.want(), kv=out)
        fa.default_workspace("cuda").check()
        s = Server(old, old, [1, 70, 2, 33], 16, pad=pad, spare=0)
        s.count -= 1                             # a page too few, for the last sequence
        d = s.device()
        d["keep"] = d["kv"]
        out = d["kv"] if place else torch.empty_like(d["kv"])
        got = step(fa, s, d, kv_len_out=out)
        with pytest.raises(fa.FAError, match="sequence 3"):
            fa.default_workspace("cuda").check()
        assert np.array_equal(out.cpu().numpy(), old) and not got[0].any()
    s = Server(old, [30, 50, 9, 0], [1, 1, 1, 1], 16)
    d = s.device()
    with pytest.raises(fa.FAError, match="overlap"):
        step(fa, s, d, kv_len_out=d["keep"])
