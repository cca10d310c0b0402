"""The paged cache held in 8 bits in use: steps of a server (fa_paged_step,
fa_kv_append_scaled, fa_fwd_paged_scaled, one after the other), and what such a
cache may hold where nobody looks.

Tolerances beside test_paged_scaled.py's: a code is off by half a step of e4m3 at
x / scale when it is written, and each time its scale grows by at most half the
smallest step, 2^-10 of the scale of that time; these scales are powers of two, so
that their sum stays below 2 x 2^-10 of the last.
"""
import numpy as np
import pytest
import torch

from block_sparse_attention_fa_gb300 import synth
from tests.test_paged import fa, reference  # noqa: F401  (fa: the fixture)
from tests.test_paged_scaled import Batch8, codes_of, compare8, half_step, run8, run_append, tables, turned
from tests.test_paged_step import plain

gpu = pytest.mark.gpu


class Loop:
    """A server of B sequences over one cache: what the device holds, and the tokens that it should hold."""

    def __init__(self, D, page, S, most, seed):
        self.r = np.random.default_rng(seed)
        self.B, self.Hq, self.Hkv, self.D, self.page, self.S, self.most = 6, 6, 2, D, page, S, most
        self.T, self.longest = self.B * most + 7, S * page + 150
        self.pages = self.B * -(-self.longest // page) + S + 3
        ids = self.r.permutation(self.pages).astype(np.int32)
        d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()   # noqa: E731
        table = np.full((self.B, -(-self.longest // page)), -1, np.int32)
        table[:, :S] = ids[:S]
        free = np.full(self.pages, -1, np.int32)
        free[:self.pages - S] = ids[S:]
        i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.free, self.count = d(table), d(free), d(np.array([self.pages - S], np.int32))
        self.kv, self.new, self.keep = i32(self.B), i32(self.B), i32(self.B)
        nan = np.full((self.pages, self.Hkv, page, D), np.nan)
        self.kc, self.vc = codes_of(nan).cuda(), codes_of(nan).cuda()
        self.s = {n: torch.full((self.pages, self.Hkv), float("nan"), device="cuda") for n in ("k_scale", "v_scale")}
        self.rot = D // 2
        self.cos, self.sin = tables(self.longest + 1, self.rot)
        self.turn = dict(cos=d(self.cos), sin=d(self.sin))
        self.x = torch.zeros((self.T, self.Hq + 2 * self.Hkv, D), dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros((self.T, self.Hq, D), dtype=torch.bfloat16, device="cuda")
        self.o, self.lse = torch.zeros_like(self.q), torch.zeros((self.T, self.Hq), device="cuda")
        self.tokens = [(np.zeros((0, self.Hkv, D)),) * 4] * self.B      # k, its rotation's magnitude, v, 0
        self.slots = [None] * 3

    def fill_prefix(self, fa):  # noqa: F811
        n = self.S * self.page
        x = synth.round_to_bf16(synth.standard_normal(3, (n, 2 * self.Hkv, self.D)))
        xd = torch.from_numpy(x).cuda().to(torch.bfloat16)
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        fa.kv_append(None, xd[:, :self.Hkv], xd[:, self.Hkv:], self.kc, self.vc, self.table[:1], i32(n), i32(0, n), **self.s,
                     **self.turn)
        self.prefix = self.token_values(x, 0)

    def token_values(self, x, first):
        ks = [turned(x[t, :self.Hkv], first + t, self.rot, False, self.cos, self.sin) for t in range(len(x))]
        k, mag = (np.array([z[e] for z in ks]).reshape(len(x), self.Hkv, self.D) for e in range(2))
        v = x[:, self.Hkv:].astype(np.float64)
        return k, mag, v, np.zeros_like(v)

    def step(self, fa, **kw):  # noqa: F811
        qs, slots, pos = fa.paged_step(self.new, self.kv, self.table, self.free, self.count, page_size=self.page,
                                       total_q=self.T, keep_len=self.keep, shared_pages=self.S, **kw)
        H, G = self.Hq, self.Hkv
        fa.kv_append(self.x[:, :H], self.x[:, H:H + G], self.x[:, H + G:], self.kc, self.vc, self.table, self.kv, qs, **self.s,
                     **self.turn, positions=pos, q_out=self.q, **kw)
        fa.fwd_paged(self.q, self.kc, self.vc, self.table, self.kv, qs, **self.s, max_q_len=self.most, mask="sink_window",
                     window=100, sinks=4, shared_len=self.S * self.page, out=self.o, lse=self.lse, **kw)
        self.slots = qs, slots, pos

    def draw(self):
        """The next step's lengths and inputs."""
        r, P = self.r, self.S * self.page
        old = self.kv.cpu().numpy().astype(np.int64)
        keep, new = old.copy(), r.integers(0, self.most + 1, self.B)
        for b in range(self.B):
            u = r.random()
            if old[b] == 0:                      # starts, or waits
                keep[b], new[b] = (P, max(new[b], 1)) if u < 0.7 else (0, 0)
            elif u < 0.1 or old[b] + self.most > self.longest:           # ends
                keep[b] = new[b] = 0
            elif u < 0.5:                        # drafts rejected
                keep[b] = max(P, old[b] - r.integers(0, 5))
        x = synth.round_to_bf16(synth.standard_normal(int(r.integers(1 << 30)), tuple(self.x.shape)) *
                                2.0 ** r.integers(-2, 2))
        self.new.copy_(torch.from_numpy(new))
        self.keep.copy_(torch.from_numpy(keep))
        self.x.copy_(torch.from_numpy(x))
        self.before = old, keep, new, x, self.table.cpu().numpy(), self.free.cpu().numpy(), self.count.item()

    def check(self):
        old, keep, new, x, table, free, count = self.before
        want = plain(old, keep, new, table, free, count, self.page, self.S, self.T)
        qs, slots, pos = self.slots
        for got, w in zip((self.kv, self.count, qs, self.table, self.free, slots, pos), want):
            assert np.array_equal(got.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
        table, at = want[3], want[2]
        codes = [z.float().double().cpu().numpy() for z in (self.kc, self.vc)]
        scale = [self.s[n].double().cpu().numpy() for n in ("k_scale", "v_scale")]
        for b in range(self.B):
            had = self.tokens[b]
            if self.S and len(had[0]) < keep[b]:
                had = self.prefix                # a sequence begins with it
            fresh = self.token_values(x[at[b]:at[b + 1], self.Hq:], keep[b])
            self.tokens[b] = tuple(np.concatenate([h[:keep[b]], f]) for h, f in zip(had, fresh))
        self.k, self.v, self.new_n, self.kv_n = [], [], list(new), list(want[0])
        for b in range(self.B):
            j = np.arange(self.kv_n[b])
            pg = table[b, j // self.page]
            for e, into in enumerate((self.k, self.v)):
                c, s = codes[e][pg, :, j % self.page], scale[e][pg][..., None]
                real, mag = self.tokens[b][2 * e:2 * e + 2]
                assert (np.abs(c * s - real) <= s * (half_step(real / s) + 2.0 ** -9) + 3 * 2.0 ** -24 * mag).all(), (b, e)
                into.append(c * s)
        q = self.q.float().cpu().numpy()
        bt = type("Seen", (), dict(new=self.new_n, kv=[int(n) for n in self.kv_n], k=self.k, v=self.v, q_start=at, total=self.T,
                                   Hkv=self.Hkv, D=self.D))
        compare8((self.o, self.lse), reference(bt, q, "sink_window", 100, 4), bt)


@gpu
@pytest.mark.parametrize("D,page,S", [(64, 16, 0), (128, 64, 0), (128, 16, 3), (64, 32, 1)])
@pytest.mark.parametrize("most", [2, 5, 40])
@pytest.mark.parametrize("how", ["eager", "captured", "stream"])
def test_serving_steps(fa, D, page, S, most, how):  # noqa: F811
    """Sequences that start, grow, have drafts rejected and end: each step's pages, codes and attention."""
    s = Loop(D, page, S, most, seed=most + page)
    if S:
        s.fill_prefix(fa)
    s.step(fa)                                   # an empty one
    assert not s.slots[0].any() and (s.slots[1] == -1).all()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if how == "captured":
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s.step(fa)
    for _ in range(14 if most < 40 else 7):
        s.draw()
        torch.cuda.synchronize()
        if how == "captured":
            g.replay()
        elif how == "stream":
            s.step(fa, stream=side)
        else:
            s.step(fa)
        torch.cuda.synchronize()
        s.check()
    fa.default_workspace("cuda").check()
    fa.default_workspace("cuda", side).check()


@gpu
@pytest.mark.parametrize("n,Hq", [(1, 2), (3, 4), (3, 8), (60, 4)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
def test_keys_that_nobody_sees(fa, n, Hq, D, page):  # noqa: F811
    """NaN codes, and scales of whole pages, outside every row's window."""
    window, sinks = 90, 5
    bt = Batch8([n, n, n], [n + 700, n + 91, n], 2, D, page, kind="any")
    for b, L in enumerate(bt.kv):
        j = np.arange(sinks, max(L - n - window, sinks))
        bt.k_codes[bt.table[b, j // page], :, j % page] = np.nan
        bt.v_codes[bt.table[b, j // page], :, j % page] = np.nan
        for e in range(-(-L // page)):
            if e * page >= sinks and (e + 1) * page <= L - n - window:
                bt.k_scale[bt.table[b, e]] = np.nan
                bt.v_scale[bt.table[b, e]] = np.inf
    run8(fa, bt, Hq, "sink_window", window, sinks)


@gpu
@pytest.mark.parametrize("n,Hq", [(1, 2), (3, 8), (60, 4)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("which", ["k", "v"])
def test_a_nan_that_is_seen_spreads(fa, n, Hq, D, which):  # noqa: F811
    bt = Batch8([n, n, n], [n + 700, n + 300, n + 5], 2, D, 32)
    getattr(bt, which + "_codes")[bt.table[1, 7], 1, 13, 40] = np.nan      # key 237
    q = bt.queries(Hq)
    dev, s = bt.device8()
    o, lse = fa.fwd_paged(torch.from_numpy(q).cuda().to(torch.bfloat16), *dev, **s, max_q_len=n)
    fa.default_workspace("cuda").check()
    hit = slice(n, 2 * n), slice(Hq // 2, Hq)
    assert o[hit][..., 40].isnan().all()
    if which == "k":
        assert o[hit].isnan().all() and lse[hit].isnan().all()
    ro, rl, A = reference(bt, q, "causal", 0, 0)
    rl[hit] = np.nan                             # (not compared)
    compare8((o, lse), (ro, rl, A), bt)


@gpu
@pytest.mark.parametrize("n,Hq", [(1, 2), (3, 8), (60, 4)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("all_pages", [False, True])
def test_scales_of_zero(fa, n, Hq, D, all_pages):  # noqa: F811
    bt = Batch8([n, n], [n + 500, n + 100], 2, D, 32, kind="any")
    for e in range(0, 18, 1 if all_pages else 3):
        for b in range(2):
            pg = bt.table[b, e] if e < bt.table.shape[1] else -1
            if pg >= 0:
                bt.k_scale[pg, 1] = bt.v_scale[pg] = 0
                bt.k[b][32 * e:32 * e + 32, 1] = 0
                bt.v[b][32 * e:32 * e + 32] = 0
    run8(fa, bt, Hq)


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_queries_of_a_wide_range(fa, D):  # noqa: F811
    """Rows whose elements are 2^-20 .. 1 of their largest, in every kernel."""
    for n in (1, 3, 60):
        bt = Batch8([n, n], [n + 500, n + 100], 2, D, 32)
        r = np.random.default_rng(n)
        q = np.copysign(2.0 ** r.uniform(-18, 2, (bt.total, 8, D)), r.normal(size=(bt.total, 8, D)))
        q = synth.round_to_bf16(q.astype(np.float32))
        most = max(np.abs(k).sum(-1).max() for k in bt.k)
        run8(fa, bt, 8, q=q, score_err=2.0 ** -18 * np.abs(q).max(-1).astype(np.float64) * most / np.sqrt(D))


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_slices_of_a_projection_and_empty_batches(fa, D):  # noqa: F811
    for n in (1, 3, 60):
        run8(fa, Batch8([n, 0, n], [n + 500, 20, n + 100], 2, D, 32, pad=3), 8, fused=True)
        run8(fa, Batch8([0, 0, 0], [500, 0, 100], 2, D, 32, pad=3), 8, max_q_len=n)


@gpu
@pytest.mark.parametrize("n", [1, 3])
def test_2048_sequences(fa, n):  # noqa: F811
    r = np.random.default_rng(n)
    kv = r.integers(n, 200, 2048)
    run8(fa, Batch8([n] * 2048, list(kv), 1, 64, 16), 4 if n == 3 else 2, max_q_len=n)


@gpu
@pytest.mark.parametrize("n,Hq", [(1, 8), (3, 32), (70, 8)])
def test_offsets_past_32_bits(fa, n, Hq):  # noqa: F811
    """Pages behind the first 4 GB of codes."""
    bt = Batch8([n, n], [n + 500, n + 300], 8, 128, 256)
    used, num = bt.k_codes.shape[0], (1 << 32) // (8 * 256 * 128) + 20
    (kc, vc, table, kv, qs), s = bt.device8()
    far = []
    for small in (kc, vc):
        t = torch.full((num, 8, 256, 128), 0x7f, dtype=torch.uint8, device="cuda")
        t[num - used:] = small.view(torch.uint8)
        far.append(t.view(torch.float8_e4m3fn))
    fars = {}
    for name, t in s.items():
        fars[name] = torch.full((num, 8), float("nan"), device="cuda")
        fars[name][num - used:] = t
    ftable = torch.where(table >= 0, table + (num - used), table)
    x = torch.randn(bt.total, Hq + 16, 128, device="cuda").to(torch.bfloat16)
    got = []
    for cache, tb, sc in (((kc, vc), table, s), (far, ftable, fars)):
        fa.kv_append(None, x[:, Hq:Hq + 8], x[:, Hq + 8:], *cache, tb, kv, qs, **sc)
        got.append(fa.fwd_paged(x[:, :Hq], *cache, tb, kv, qs, **sc, max_q_len=n))
    fa.default_workspace("cuda").check()
    for a, b in zip(*got):
        assert torch.equal(a, b)
    for a, b in zip((kc, vc), far):
        assert torch.equal(a.view(torch.uint8), b[num - used:].view(torch.uint8))
        assert (b[:num - used].view(torch.uint8) == 0x7f).all()


@gpu
def test_slots_past_32_bits(fa):  # noqa: F811
    first = (1 << 31) // 256 + 5
    free = torch.arange(first, first + 4, dtype=torch.int32, device="cuda")
    free = torch.cat([free, torch.zeros(first, dtype=torch.int32, device="cuda")])
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, kv = torch.full((1, 3), -1, dtype=torch.int32, device="cuda"), i32(0)
    _, slots, _ = fa.paged_step(i32(300), kv, table, free, i32(4), page_size=256, total_q=301)
    fa.default_workspace("cuda").check()
    want = np.concatenate([(first + 3) * 256 + np.arange(256), (first + 2) * 256 + np.arange(44), [-1]])
    assert np.array_equal(slots.cpu().numpy(), want)


@gpu
def test_graphs_on_two_streams(fa):  # noqa: F811
    """Captured calls of two batches, replayed side by side, give what each gives alone."""
    batches = [Batch8([1] * 40, list(np.random.default_rng(e).integers(1, 900, 40)), 2, 64, 16, seed=e) for e in range(2)]
    graphs, outs, want = [], [], []
    streams = [torch.cuda.Stream() for _ in batches]
    for bt, st in zip(batches, streams):
        dev, s = bt.device8()
        q = torch.from_numpy(bt.queries(8)).cuda().to(torch.bfloat16)
        want.append(fa.fwd_paged(q, *dev, **s, max_q_len=1))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(fa.fwd_paged(q, *dev, **s, max_q_len=1))
        graphs.append((g, dev, s, q))
    for _ in range(20):
        for (g, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
def test_what_a_cache_may_be(fa):  # noqa: F811
    """A bf16 cache has no scales, one of 8 bits has both, one per page and kv head."""
    bt = Batch8([1], [20], 2, 64, 16)
    dev, s = bt.device8()
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    plain_cache = bt.device()

    def both(cache, **kw):
        for call in (lambda: fa.fwd_paged(q, *cache, **kw), lambda: fa.kv_append(None, q[:, :2], q[:, 2:], *cache, **kw)):
            with pytest.raises(ValueError):
                call()

    both(plain_cache, **s)
    both(dev)
    both(dev, k_scale=s["k_scale"])
    both(dev, v_scale=s["v_scale"])
    both((dev[0], plain_cache[1], *dev[2:]), **s)
    both(dev, k_scale=s["k_scale"], v_scale=s["v_scale"][:-1])
    both(dev, k_scale=s["k_scale"].double(), v_scale=s["v_scale"])
    both(dev, k_scale=s["k_scale"].t().contiguous().t(), v_scale=s["v_scale"])
    both(dev, k_scale=s["k_scale"].cpu(), v_scale=s["v_scale"])


@gpu
@pytest.mark.parametrize("n,Hq", [(1, 2), (3, 8), (60, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_that_several_sequences_name(fa, n, Hq, D):  # noqa: F811
    """A prefix read through every sequence's own row of the table."""
    bt = Batch8([n, n, n], [n + 400, n + 330, n + 320], 2, D, 32, shared=320, kind="any")
    bt.shared = 0
    run8(fa, bt, Hq)


@gpu
@pytest.mark.parametrize("n,Hq", [(1, 2), (3, 8), (60, 4)])
@pytest.mark.parametrize("shared", [0, 64])
def test_bad_sequences_are_reported(fa, n, Hq, shared):  # noqa: F811
    """More new tokens than max_q_len, a page that is not there: a status, and the others' rows as they should be."""
    bt = Batch8([n, n + 1, n, n], [n + 100 + shared, n + 90 + shared, n + 80 + shared, n + 70 + shared], 2, 64, 16, shared=shared)
    q = bt.queries(Hq)
    dev, s = bt.device8()
    dev[2][2, (bt.kv[2] - 1) // 16] = 1 << 30
    o, lse = fa.fwd_paged(torch.from_numpy(q).cuda().to(torch.bfloat16), *dev, **s, max_q_len=n, shared_len=shared)
    with pytest.raises(fa.FAError) as e:
        fa.default_workspace("cuda").check()
    assert e.value.status == fa.ERR_DEVICE_CHECK
    ro, rl, A = reference(bt, q, "causal", 0, 0)
    rl[bt.q_start[1]:bt.q_start[3]] = np.nan     # (not compared)
    compare8((o, lse), (ro, rl, A), bt)


@gpu
def test_append_without_a_prompt_then_read_far_apart(fa):  # noqa: F811
    """An append of prompts of every length, then attention over just them."""
    new = [1, 15, 16, 17, 33, 200]
    for page in (16, 64):
        bt = Batch8(new, new, 2, 128, page)
        run_append(fa, bt, synth.round_to_bf16(synth.standard_normal(9, (bt.total, 10, 128))), 6, 128, False, *tables(201, 128))
