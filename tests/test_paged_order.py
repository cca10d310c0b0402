"""Steps of a serving loop over a shared prefix one right behind the other, in one
captured graph: the lengths, the page table and the rows change before every
step, and every step reads what the one before it has appended.  The prefix's
kernel and the sequences' own overlap; each has to see all of it.
"""
import pytest
import torch

from tests.test_paged import Batch, compare, fa, reference  # noqa: F401  (fa: the fixture)

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("shared", [64, 1000])
def test_steps_in_a_graph(fa, shared, n, D):  # noqa: F811
    Hq, Hkv, page, B, steps = 8, 2, 16, 6, 8
    bt = Batch([n] * B, [shared + 60 + 50 * b + n * steps for b in range(B)], Hkv, D, page, shared=shared)
    kc0, vc0, table0, kv0, qs = bt.device()
    kc0, vc0 = kc0.nan_to_num(0.5), vc0.nan_to_num(0.5)
    # step s: every sequence n longer, its pages those of the one b + s places on
    lens = torch.stack([torch.tensor([bt.kv[(b + s) % B] - n * (steps - 1 - s) for b in range(B)]) for s in range(steps)])
    lens = lens.to(torch.int32).cuda()
    tables = torch.stack([table0.roll(-s, 0) for s in range(steps)])
    gen = torch.Generator(device="cuda").manual_seed(3)
    rows = torch.randn(steps, B * n, Hq + 2 * Hkv, D, generator=gen, device="cuda").to(torch.bfloat16)
    angle = torch.rand(2000 + shared, D // 2, generator=gen, device="cuda") * 6
    kw = dict(cos=angle.cos(), sin=angle.sin())

    def run(between):
        kc, vc, table, kv = kc0.clone(), vc0.clone(), torch.full_like(table0, -1), torch.zeros_like(kv0)
        x = torch.zeros_like(rows[0])
        got = []
        for s in range(steps):
            between()
            kv.copy_(lens[s])
            table.copy_(tables[s])
            x.copy_(rows[s])
            q = fa.kv_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, table, kv, qs, **kw)
            # attention twice: behind an append, and behind a call of its own kind
            got += [fa.fwd_paged(q, kc, vc, table, kv, qs, max_q_len=n, shared_len=shared),
                    fa.fwd_paged(q + 0, kc, vc, table, kv, qs, max_q_len=n, shared_len=shared),
                    fa.fwd_paged(q, kc, vc, table, kv, qs, max_q_len=n, shared_len=shared)]
        return got, kc, vc

    want, wk, wv = run(torch.cuda.synchronize)
    fa.default_workspace("cuda").check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got, gk, gv = run(lambda: torch.cuda._sleep(20000))
    for _ in range(5):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(gk, wk) and torch.equal(gv, wv)
        for (o, lse), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)


@gpu
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("fill", ["zeros", "ones", "mark"])
def test_scratch_may_hold_anything(fa, n, fill):  # noqa: F811
    """Also the mark that the prefix's kernel leaves for the sequences' own, which is gone after the call."""
    bt = Batch([n, n], [400 + n, 300 + n], 2, 64, 16, shared=256)
    dev, q = bt.device(), torch.from_numpy(bt.queries(4)).cuda().to(torch.bfloat16)
    scratch = fa.paged_scratch(q, *dev, max_q_len=n, shared_len=256)
    scratch.fill_({"zeros": 0, "ones": 255, "mark": 0}[fill])
    if fill == "mark":
        mark = 0x9d3ac1f05b7e2468
        scratch[8:16] = torch.tensor([(mark >> 8 * k) & 255 for k in range(8)], dtype=torch.uint8, device="cuda")
    for _ in range(2):
        got = fa.fwd_paged(q, *dev, max_q_len=n, shared_len=256, scratch=scratch)
        fa.default_workspace("cuda").check()
        compare(got, reference(bt, bt.queries(4), "causal", 0, 0))
        assert (scratch[8:16] == 0).all()
