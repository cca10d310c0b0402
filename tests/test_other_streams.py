"""Calls on a stream that is not the current one: what they allocate (outputs,
BlockMasks, scratch) is that stream's memory, not memory which the current
stream has just given back and may still be writing.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _inputs(T, Hq, Hkv, D, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda h: torch.randn(1, h, T, D, generator=gen, device="cuda").to(torch.bfloat16)   # noqa: E731
    return rand(Hq), rand(Hkv), rand(Hkv), rand(Hq), rand(Hq)[:, :, :8].contiguous()


def _step(x, **kw):
    from block_sparse_attention_fa_gb300 import fa
    q, k, v, g, q8 = x
    T = q.shape[2]
    bm = fa.block_mask("sink_window", 1, 1, T, T, window=100, sinks=4, device="cuda", **kw)
    o, lse = fa.fwd(q, k, v, bm, **kw)
    first = fa.block_mask("sink_window", 1, 1, 8, T, window=100, sinks=4, device="cuda", **kw)
    few = fa.fwd_decode(q8, k, v, first, **kw)
    grads = fa.bwd(q, k, v, o, lse, g, bm, **kw)
    return (o, lse, *grads, *few, bm.kv_indices, bm.full_kv_num_blocks, *bm.cols(**kw).values())


def test_memory_is_the_streams_own():
    x = _inputs(700, 4, 2, 64, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    held = [torch.empty_like(t) for t in _step(x) for _ in range(4)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in held]
    del held
    got = _step(x, stream=side)
    for t in got:
        assert not any(a <= t.data_ptr() < b for a, b in spans)
    torch.cuda.synchronize()


def test_a_busy_current_stream_does_not_write_them():
    """Blocks that the current stream gives back and is still to fill."""
    x = _inputs(700, 4, 2, 64, 2)
    side = torch.cuda.Stream()
    want = _step(x)
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda._sleep(30_000_000)
        for t in [torch.empty_like(t) for t in want for _ in range(4)]:
            t.fill_(77)
        del t
        got = _step(x, stream=side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
