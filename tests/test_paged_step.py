"""fa_paged_step: a step's pages, offsets and slots from its sequences' lengths,
against the definition carried out request by request.  Whole numbers: every
comparison is for equality."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_paged import FAKE, fa  # noqa: F401  (fa: the fixture)

gpu = pytest.mark.gpu


def plain(old, keep, new, table, free, count, page, shared, total):
    """The definition, one sequence and one page after the other."""
    table, free = table.copy(), free.copy()
    had = [max(-(-int(x) // page), shared) for x in old]
    has = [max(-(-int(k + n) // page), shared) for k, n in zip(keep, new)]
    for b in reversed(range(len(old))):
        for e in reversed(range(has[b], had[b])):
            free[count] = table[b, e]
            count += 1
    start, slots, places = [0], np.full(total, -1, np.int64), np.zeros(total, np.int32)
    for b in range(len(old)):
        for e in range(had[b], has[b]):
            count -= 1
            table[b, e] = free[count]
        at = keep[b] + np.arange(new[b])
        rows = slice(start[-1], start[-1] + new[b])
        slots[rows] = table[b, at // page].astype(np.int64) * page + at % page
        places[rows] = at
        start.append(start[-1] + int(new[b]))
    return np.array(keep) + new, count, np.array(start), table, free, slots, places


class Server:
    """Sequences of `old` tokens on shuffled pages, `spare` pages free beside those that the step needs."""

    def __init__(self, old, keep, new, page, shared=0, pad=0, spare=3, seed=0, first=0):
        self.old, self.keep, self.new = (np.asarray(x, np.int64) for x in (old, keep, new))
        self.page, self.shared, self.total = page, shared, int(self.new.sum()) + pad
        B = len(old)
        had = np.maximum(-(-self.old // page), shared)
        has = np.maximum(-(-(self.keep + self.new) // page), shared)
        need = int(np.maximum(has - had, 0).sum() - np.maximum(had - has, 0).sum())
        used = int((had - shared).sum()) + shared
        n = max(used + max(need, 0) + spare, 1)  # (a server has pages)
        ids = (first + np.random.default_rng(seed).permutation(n)).astype(np.int32)
        self.table = np.full((B, max(int(max(had.max(), has.max())), 1) + 1), -1, np.int32)
        self.table[:, :shared] = ids[:shared]
        at = shared
        for b in range(B):
            self.table[b, shared:had[b]] = ids[at:at + had[b] - shared]
            at += had[b] - shared
        self.count = n - at
        self.free = np.full(n + first, -7, np.int32)
        self.free[:self.count] = ids[at:]

    def device(self):
        d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda().to(torch.int32)   # noqa: E731
        return dict(new=d(self.new), kv=d(self.old), table=d(self.table), free=d(self.free), count=d(np.array([self.count])),
                    keep=d(self.keep))

    def want(self):
        return plain(self.old, self.keep, self.new, self.table, self.free, self.count, self.page, self.shared, self.total)


def step(fa, s, d, **kw):  # noqa: F811
    got = fa.paged_step(d["new"], d["kv"], d["table"], d["free"], d["count"], page_size=s.page, total_q=s.total,
                        keep_len=d["keep"], shared_pages=s.shared, **kw)
    return got


def same(d, got, want, kv=None, count=None):
    kv, count = d["kv"] if kv is None else kv, d["count"] if count is None else count
    for x, y in zip((kv, count, got[0], d["table"], d["free"], got[1], got[2]), want):
        assert np.array_equal(x.cpu().numpy().reshape(-1), np.asarray(y).reshape(-1))


def mixed(B, page, seed, longest=3000, prompt=900, shared=0):
    r = np.random.default_rng(seed)
    old = shared * page + r.integers(0, longest, B)
    keep, new = old - np.minimum(r.integers(0, 6, B), old - shared * page), r.integers(0, 5, B)
    u = r.random(B)
    old[u < 0.3] = 0
    keep[u < 0.3] = shared * page
    new[u < 0.3] = r.integers(1, prompt, (u < 0.3).sum())
    keep[u > 0.85] = 0
    new[u > 0.85] = 0
    return old, keep, new


# ------------------------------------------------------------------ CPU: refusals
def _args(fa, **kw):  # noqa: F811
    a = fa.PagedStepArgs()
    a.B, a.num_pages, a.page_size, a.max_pages, a.shared_pages, a.total_q = 4, 32, 16, 8, 0, 10
    names = [f[0] for f in fa.PagedStepArgs._fields_[6:]]
    for e, name in enumerate(names):
        setattr(a, name, FAKE + 4096 * e)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(total_q=-1), 1), (dict(B=2049), 2),
    (dict(page_size=24), 2), (dict(page_size=8), 2), (dict(page_size=512), 2), (dict(max_pages=2**31 - 1), 2),
    (dict(shared_pages=-1), 1), (dict(shared_pages=9), 1), (dict(new_len=None), 1), (dict(kv_len=None), 1),
    (dict(page_table=None), 1), (dict(free_pages=None), 1), (dict(free_count=None), 1), (dict(kv_len_out=None), 1),
    (dict(free_count_out=None), 1), (dict(q_start=None), 1), (dict(keep_len=FAKE + 2), 1), (dict(slots=FAKE + 4), 1),
    (dict(positions=FAKE + 1), 1), (dict(page_table=FAKE), 1), (dict(q_start=FAKE + 8), 1),
    (dict(slots=FAKE + 3 * 4096), 1), (dict(kv_len_out=FAKE + 2 * 4096 + 4), 1)], ids=str)
def test_refusals(fa, kw, status):  # noqa: F811
    lib = fa.load_library()
    assert lib.fa_paged_step(ctypes.byref(_args(fa, **kw)), FAKE, None) == status, lib.fa_last_error()
    assert lib.fa_last_error()


def test_refuses_null(fa):  # noqa: F811
    lib = fa.load_library()
    assert lib.fa_paged_step(None, FAKE, None) == fa.ERR_INVALID_ARG
    assert lib.fa_paged_step(ctypes.byref(_args(fa)), None, None) == fa.ERR_INVALID_ARG
    assert fa._PAGED_STEP.size == ctypes.sizeof(fa.PagedStepArgs)
    n = len(fa.PagedStepArgs._fields_)
    s = fa.PagedStepArgs.from_buffer_copy(fa._PAGED_STEP.pack(*range(1, n + 1)))
    assert [getattr(s, f[0]) for f in s._fields_] == list(range(1, n + 1))


def test_binding_refuses_on_the_cpu(fa):  # noqa: F811
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA int32"):
        fa.paged_step(t, t, t.view(4, 1), t, t[:1], page_size=16, total_q=4)


# ------------------------------------------------------------------ GPU
@gpu
@pytest.mark.parametrize("page", [16, 32, 256])
@pytest.mark.parametrize("B,shared,pad", [(1, 0, 0), (5, 0, 2), (64, 3, 0), (300, 0, 5000), (2048, 1, 1)])
def test_mixed_steps(fa, B, page, shared, pad):  # noqa: F811
    s = Server(*mixed(B, page, B + page, shared=shared), page, shared, pad)
    d = s.device()
    want = s.want()
    # beside the lengths and the count before: the call may be repeated
    kv, count = torch.full_like(d["kv"], 99), torch.full_like(d["count"], 99)
    for _ in range(2):
        got = step(fa, s, d, kv_len_out=kv, free_count_out=count)
        same(d, got, want, kv, count)
    assert np.array_equal(d["kv"].cpu().numpy(), s.old) and d["count"].item() == s.count
    # in place
    d = s.device()
    same(d, step(fa, s, d), want)
    fa.default_workspace("cuda").check()


@gpu
@pytest.mark.parametrize("old,keep,new", [
    ([0], [0], [1]), ([16], [16], [1]), ([15], [15], [1]), ([17], [17], [0]), ([17], [16], [0]), ([16], [0], [0]),
    ([0, 0], [0, 0], [0, 0]), ([33, 0, 16], [16, 0, 16], [1, 40, 16]), ([100, 5], [0, 5], [0, 200])])
def test_borders(fa, old, keep, new):  # noqa: F811
    s = Server(old, keep, new, 16, spare=0)
    d = s.device()
    same(d, step(fa, s, d), s.want())
    fa.default_workspace("cuda").check()


@gpu
def test_all_kept_and_no_rows(fa):  # noqa: F811
    s = Server([30, 64], [30, 64], [2, 1], 16, pad=4)
    d = s.device()
    got = fa.paged_step(d["new"], d["kv"], d["table"], d["free"], d["count"], page_size=16, total_q=s.total)
    same(d, got, s.want())
    s = Server([30, 64], [3, 0], [0, 0], 16)
    d = s.device()
    got = step(fa, s, d)
    assert got[1].numel() == got[2].numel() == 0
    same(d, got, s.want())
    # without slots or positions, through the C ABI
    s = Server([30, 64], [30, 64], [2, 1], 16)
    d = s.device()
    q = torch.zeros(3, dtype=torch.int32, device="cuda")
    a = fa.PagedStepArgs(2, s.free.size, 16, s.table.shape[1], 0, s.total, d["new"].data_ptr(), None, d["kv"].data_ptr(),
                         d["table"].data_ptr(), d["free"].data_ptr(), d["count"].data_ptr(), d["kv"].data_ptr(),
                         d["count"].data_ptr(), q.data_ptr(), None, None)
    ws = fa.default_workspace("cuda")
    assert fa.load_library().fa_paged_step(ctypes.byref(a), ws.tensor.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    ws.check()
    w = s.want()
    same(d, (q, torch.from_numpy(w[5]), torch.from_numpy(w[6])), w)


@gpu
def test_giving_back_undoes_taking(fa):  # noqa: F811
    s = Server([0, 40, 7], [0, 40, 7], [100, 30, 3], 16, spare=5)
    d = s.device()
    before = d["free"].clone()
    step(fa, s, d)
    back = torch.tensor([0, 40, 7], dtype=torch.int32, device="cuda")
    none = torch.zeros_like(back)
    fa.paged_step(none, d["kv"], d["table"], d["free"], d["count"], page_size=16, total_q=0, keep_len=back)
    assert torch.equal(d["kv"], back) and d["count"].item() == s.count and torch.equal(d["free"], before)
    fa.default_workspace("cuda").check()


BAD = {
    "negative new_len": dict(new=[1, -1, 2]), "negative keep_len": dict(keep=[20, -3, 9]),
    "keep_len past the cache": dict(keep=[20, 51, 9]), "past the row of the table": dict(new=[1, 10000, 2]),
    "negative kv_len": dict(old=[20, -5, 9]), "rows": dict(total=2), "pages": dict(count=0),
    "count past the stack": dict(count=10**6), "negative count": dict(count=-1),
    "more given back than the stack holds": dict(full=True), "new_len adds up past 32 bits": dict(new=[2**30, 2**30, 2**30], total=2**20)}


@gpu
@pytest.mark.parametrize("what", BAD, ids=lambda s: s.replace(" ", "_"))
@pytest.mark.parametrize("pad", [0, 6000])
def test_steps_that_cannot_be_made(fa, what, pad):  # noqa: F811
    # sequence 0 needs a page, sequence 1 gives one back and sequence 2 neither
    s = Server([32, 50, 9], [32, 40, 9], [1, 1, 2], 16, pad=pad, spare=2)
    kw = BAD[what]
    for k in ("new", "keep", "old"):
        if k in kw:
            setattr(s, k, np.array(kw[k]))
    if "total" in kw:
        s.total = kw["total"]
    if "count" in kw:
        s.count = kw["count"]
        if kw["count"] == 0:
            s.keep[1] = 50                       # none given back either
    if "full" in kw:
        s.count, s.keep[0] = s.free.size, 31
    d = s.device()
    before = {k: v.clone() for k, v in d.items()}
    kv, count = torch.full_like(d["kv"], 99), torch.full_like(d["count"], 99)
    got = step(fa, s, d, kv_len_out=kv, free_count_out=count)
    with pytest.raises(fa.FAError) as e:
        fa.default_workspace("cuda").check()
    assert e.value.status == fa.ERR_DEVICE_CHECK
    assert all(torch.equal(d[k], v) for k, v in before.items())
    assert torch.equal(kv, d["kv"]) and torch.equal(count, d["count"])
    assert not got[0].any() and (got[1] == -1).all() and not got[2].any()
    fa.default_workspace("cuda").check()


@gpu
@pytest.mark.parametrize("pad", [0, 6000])
@pytest.mark.parametrize("which", ["free", "given", "kept"])
def test_bad_pages_are_reported(fa, which, pad):  # noqa: F811
    s = Server([32, 50, 9], [32, 40, 9], [1, 1, 2], 16, pad=pad, spare=2)
    if which == "free":
        s.keep[1], s.free[s.count - 1] = 50, 10**6       # the page that sequence 0 takes
    if which == "given":
        s.table[1, 3] = -4                               # given back by sequence 1, taken by sequence 0
    if which == "kept":
        s.table[2, 0] = 10**6                            # of sequence 2's rows
    d = s.device()
    got = step(fa, s, d)
    with pytest.raises(fa.FAError) as e:
        fa.default_workspace("cuda").check()
    assert e.value.status == fa.ERR_DEVICE_CHECK
    kv, count, start, table, free, slots, places = s.want()
    page = slots // 16
    slots = np.where((page < 0) | (page >= s.free.size), -1, slots)
    same(d, got, (kv, count, start, table, free, slots, places))
    fa.default_workspace("cuda").check()


@gpu
def test_a_captured_step_follows_its_inputs(fa):  # noqa: F811
    page, B = 16, 40
    s = [Server(*mixed(B, page, k, 500, 300), page, pad=0, spare=50, seed=k) for k in range(3)]
    total, width, pages = (max(f(x) for x in s) for f in (lambda x: x.total, lambda x: x.table.shape[1], lambda x: x.free.size))
    for x in s:
        x.total = total
        x.table = np.pad(x.table, ((0, 0), (0, width - x.table.shape[1])), constant_values=-1)
        x.free = np.pad(x.free, (0, pages - x.free.size), constant_values=-7)
    d = s[0].device()
    step(fa, s[0], d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(fa, s[0], d)
    for x in s + s:
        for k, v in x.device().items():
            d[k].copy_(v)
        g.replay()
        same(d, got, x.want())
    fa.default_workspace("cuda").check()


@gpu
def test_on_another_stream(fa):  # noqa: F811
    s = Server(*mixed(64, 16, 5), 16)
    d = s.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(fa, s, d, stream=side)
    side.synchronize()
    same(d, got, s.want())
    fa.default_workspace("cuda", side).check(side)
