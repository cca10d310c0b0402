"""Cases, plain forms and exact values of the operators of an 8-bit paged cache.

Three operators, in the order in which a serving loop uses them: the step's page tables, offsets and slot maps from the
requests' lengths; appending rotated keys and values to a cache held in 8 bits (e4m3) with a scale for each page and kv
head; attention over that cache.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
ROPE_BASE = 10000.0
E4M3_MAX = 448.0
# scales that an append chooses: powers of two between these exponents
SCALE_EXP = (-100, 119)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of 64 requests: a few need a page, none ends; latency
        dict(name="step_decode", op="step", B=64, prompt=1, kv_len=2048, page=16, fresh=0.0, ended=0.0, drafts=1, pad=0,
             shared=0),
        # continuous batching: prompts come in, requests end and give their pages back, drafts are rejected
        dict(name="step_mixed", op="step", B=256, prompt=2000, kv_len=8192, page=32, fresh=0.2, ended=0.1, drafts=4,
             pad=100, shared=3),
        # the prompts of a large batch at once
        dict(name="step_prompts", op="step", B=512, prompt=4096, kv_len=1024, page=64, fresh=0.9, ended=0.02, drafts=1,
             pad=0, shared=0),
        # one decoding step of 64 sequences: every token joins a page that has earlier ones
        dict(name="append8_step", op="append", B=64, q_len=1, kv_len=1024, Hq=32, Hkv=8, D=128, page=16, rot=128,
             interleaved=False, ragged=True, pad=0),
        # ragged prompts, interleaved pairs, half of the head rotated, rows of padding behind the last prompt
        dict(name="append8_prompts", op="append", B=8, q_len=4096, kv_len=4096, Hq=32, Hkv=8, D=128, page=64, rot=64,
             interleaved=True, ragged=True, pad=37),
        # one user, a short context: latency
        dict(name="paged8_one", op="paged", B=1, q_len=1, kv_len=520, Hq=32, Hkv=8, D=128, page=16, window=-1, sinks=0,
             ragged=False, shared=0, cap=0.0, calibrated=False),
        # long contexts of equal length, one token each
        dict(name="paged8_long", op="paged", B=8, q_len=1, kv_len=32768, Hq=32, Hkv=8, D=128, page=64, window=-1,
             sinks=0, ragged=False, shared=0, cap=0.0, calibrated=False),
        # many ragged chats, scores capped, scales from a calibration (no powers of two), heads of 64 columns
        dict(name="paged8_chats", op="paged", B=128, q_len=1, kv_len=4096, Hq=32, Hkv=8, D=64, page=16, window=-1,
             sinks=0, ragged=True, shared=0, cap=30.0, calibrated=True),
        # streaming: ragged contexts, 3 tokens to verify each, window and sinks
        dict(name="paged8_stream", op="paged", B=64, q_len=3, kv_len=16384, Hq=16, Hkv=4, D=64, page=16, window=1024,
             sinks=4, ragged=True, shared=0, cap=0.0, calibrated=False),
        # the second chunk of long prompts
        dict(name="paged8_chunk", op="paged", B=4, q_len=1024, kv_len=8192, Hq=32, Hkv=8, D=128, page=128, window=-1,
             sinks=0, ragged=True, shared=0, cap=0.0, calibrated=False),
        # 64 chats over one long system prompt, one token each
        dict(name="shared8_chat", op="paged", B=64, q_len=1, kv_len=512, Hq=32, Hkv=8, D=128, page=64, window=-1,
             sinks=0, ragged=True, shared=16384, cap=0.0, calibrated=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "append", "paged", "paged", "shared"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "step":
        prompt = _log_int(rng, 1, 4096)
        return dict(op="step", B=_log_int(rng, 1, max(2, min(512, 800000 // prompt))), prompt=prompt,
                    kv_len=_log_int(rng, 1, 16000), page=page, fresh=rng.choice([0.0, 0.1, 0.5, 0.9]),
                    ended=rng.choice([0.0, 0.1, 0.3]), drafts=rng.randint(1, 8), pad=rng.choice([0, rng.randint(1, 300)]),
                    shared=rng.choice([0, 0, rng.randint(1, 5)]))
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    window = rng.choice([-1, -1, _log_int(rng, 1, 4096)])
    sinks = rng.choice([0, 1, 4, _log_int(rng, 1, 300)])
    if op == "append":
        n = _log_int(rng, 1, 2000)
        return dict(op="append", B=_log_int(rng, 1, max(2, min(128, 16000 // n))), q_len=n,
                    kv_len=n + _log_int(rng, 1, 2000), Hq=Hkv * group, Hkv=Hkv, D=D, page=page,
                    rot=rng.choice([32, 64, D]), interleaved=rng.random() < 0.5, ragged=rng.random() < 0.7,
                    pad=rng.randint(0, 9))
    more = dict(cap=rng.choice([0.0, 0.0, 30.0]), calibrated=rng.random() < 0.5)
    if op == "shared":
        n = rng.choice([1, 1, 2, 4, 7])
        return dict(op="paged", B=_log_int(rng, 2, 64), q_len=n, kv_len=n + _log_int(rng, 1, 700), Hq=Hkv * group,
                    Hkv=Hkv, D=D, page=page, window=window, sinks=sinks, ragged=True,
                    shared=page * rng.randint(1, max(1, _log_int(rng, 300, 16000) // page)), **more)
    n = rng.choice([1, 1, 2, 5, _log_int(rng, 1, 1000)])
    kv = n + _log_int(rng, 1, 30000 if n < 8 else 6000)
    most = max(1, min(128, 250000 // kv, 80000 // (n * Hkv * group)))
    return dict(op="paged", B=_log_int(rng, 1, most), q_len=n, kv_len=kv, Hq=Hkv * group, Hkv=Hkv, D=D, page=page,
                window=window, sinks=sinks, ragged=rng.random() < 0.7, shared=0, **more)


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dtype)


def _requests(case):
    """Old, kept and new lengths of every request: part of the case, the same for every seed."""
    r = np.random.RandomState(7 * case["B"] + case["kv_len"])
    B, front = case["B"], case["shared"] * case["page"]
    old = front + r.randint(max(1, case["kv_len"] // 8), case["kv_len"] + 1, B)
    keep, new = old.copy(), r.randint(1, case["drafts"] + 1, B)
    back = np.minimum(r.randint(0, case["drafts"], B), old - front)      # rejected drafts
    keep -= back
    u = r.random_sample(B)
    fresh, ended = u < case["fresh"], u > 1 - case["ended"]
    old[fresh] = 0                                   # not in the cache yet, beside the shared pages
    keep[fresh] = front
    new[fresh] = r.randint(max(1, case["prompt"] // 4), case["prompt"] + 1, B)[fresh]
    keep[ended] = new[ended] = 0
    return old, keep, new


def _page_counts(case, old, keep, new):
    P, S = case["page"], case["shared"]
    return np.maximum(-(-old // P), S), np.maximum(-(-(keep + new) // P), S)


def _lengths(case):
    """New tokens and cached length (new tokens included, shared prefix excluded) of every sequence: part of the
    case, the same for every seed."""
    r = np.random.RandomState(1000 * case["B"] + case["kv_len"])
    B, n, L = case["B"], case["q_len"], case["kv_len"]
    if not case["ragged"]:
        return np.full(B, n), np.full(B, L)
    new = r.randint(max(1, n // 2), n + 1, B)
    new[r.randint(B)] = n
    past = r.randint((L - n) // 8, L - n + 1, B)
    past[r.randint(B)] = L - n
    return new, new + past


def _pages(case, new, kv, gen):
    """Page table, lengths and offsets on the device; sequences own their pages, a shared prefix is stored once."""
    page, shared = case["page"], case.get("shared", 0)
    nsh = shared // page
    own_pages = -(-kv // page)
    width = int(nsh + own_pages.max())
    total = int(nsh + own_pages.sum())
    perm = torch.randperm(total, generator=gen, device=DEVICE, dtype=torch.int32)
    first = torch.from_numpy(np.concatenate([[0], np.cumsum(own_pages)[:-1]])).to(DEVICE) + nsh
    count = torch.from_numpy(own_pages).to(DEVICE)
    c = torch.arange(width, device=DEVICE)
    at = torch.where(c[None] < nsh, c[None], first[:, None] + c[None] - nsh)
    used = c[None] < nsh + count[:, None]
    table = torch.where(used, perm[at.clamp(max=total - 1)], torch.full_like(perm[:1], -1)).to(torch.int32).contiguous()
    start = np.concatenate([[0], np.cumsum(new)])
    return dict(page_table=table, num_pages=total, kv_len=torch.from_numpy(kv + shared).to(DEVICE, torch.int32),
                q_start=torch.from_numpy(start).to(DEVICE, torch.int32), rows=int(start[-1]), longest=int(kv.max()))


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, its exponent within SCALE_EXP."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)            # 448 = 0.875 2^9
    e = torch.where(amax > 0, e, torch.full_like(e, SCALE_EXP[0])).clamp(*SCALE_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _cache8(gen, shape, calibrated):
    """A cache in use: e4m3 codes and a scale for each page and kv head; heads and pages differ in size."""
    x = torch.randn(shape, generator=gen, device=DEVICE)
    x *= torch.exp(0.4 * torch.randn(shape[:2], generator=gen, device=DEVICE))[:, :, None, None]
    amax = x.abs().amax((2, 3))
    scale = amax / E4M3_MAX if calibrated else _pow2_scale(amax)
    return (x / scale[:, :, None, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    if case["op"] == "step":
        return _prepare_step(case, gen)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    new, kv = _lengths(case)
    s = dict(case=case, **_pages(case, new, kv, gen), max_q=case["q_len"])
    shape = (s["num_pages"], Hkv, case["page"], D)
    s["k_cache"], s["k_scale"] = _cache8(gen, shape, case.get("calibrated", False))
    s["v_cache"], s["v_scale"] = _cache8(gen, shape, case.get("calibrated", False))
    if case["op"] == "paged":
        s["q"] = _normal(gen, (s["rows"], Hq, D))
        return s
    total = s["rows"] + case["pad"]
    # queries, keys and values as one projection gives them
    qkv = _normal(gen, (total, (Hq + 2 * Hkv) * D))
    s["q"] = qkv[:, : Hq * D].view(total, Hq, D)
    s["k"] = qkv[:, Hq * D: (Hq + Hkv) * D].view(total, Hkv, D)
    s["v"] = qkv[:, (Hq + Hkv) * D:].view(total, Hkv, D)
    s["q_out"] = torch.zeros((total, Hq, D), dtype=torch.bfloat16, device=DEVICE)
    half = case["rot"] // 2
    freq = ROPE_BASE ** (-torch.arange(half, device=DEVICE, dtype=torch.float64) / half)
    angle = torch.arange(case["kv_len"], device=DEVICE, dtype=torch.float64)[:, None] * freq
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    return s


def _prepare_step(case, gen):
    old, keep, new = _requests(case)
    before, after = _page_counts(case, old, keep, new)
    width, S = int(max(before.max(), after.max())), case["shared"]
    used, need = int((before - S).sum()), int(np.maximum(after - before, 0).sum())
    num_pages = S + used + need + 50
    perm = torch.randperm(num_pages, generator=gen, device=DEVICE, dtype=torch.int32)
    first = torch.from_numpy(S + np.concatenate([[0], np.cumsum(before - S)[:-1]])).to(DEVICE)
    c = torch.arange(width, device=DEVICE)
    at = torch.where(c[None] < S, c[None], first[:, None] + c[None] - S).clamp(max=num_pages - 1)
    table = torch.where(c[None] < torch.from_numpy(before).to(DEVICE)[:, None], perm[at], torch.full_like(perm[:1], -1))
    free = torch.zeros(num_pages, dtype=torch.int32, device=DEVICE)
    count = num_pages - S - used
    free[:count] = perm[S + used:]
    to = lambda x: torch.from_numpy(np.asarray(x)).to(DEVICE, torch.int32)   # noqa: E731
    total = int(new.sum()) + case["pad"]
    return dict(case=case, kv_len=to(old), keep=to(keep), new=to(new), page_table=table.contiguous(), free=free,
                count=to([count]), total=total, kv_out=to(old), count_out=to([count]),
                q_start=to(np.zeros(case["B"] + 1)), slots=torch.zeros(total, dtype=torch.int64, device=DEVICE),
                positions=to(np.zeros(total)))


# --------------------------------------------------------------- operators
def run(state):
    op = state["case"]["op"]
    if op == "step":
        return _step_own(state) if own else _step_plain(state)
    if op == "append":
        return _append_own(state) if own else _append_plain(state)
    return _paged_own(state) if own else _paged_plain(state)


def _step_own(s):
    from block_sparse_attention_fa_gb300 import fa
    c = s["case"]
    # the lengths and the count before the step stay with the caller (two buffers, as graphs use them in turn)
    fa.paged_step(s["new"], s["kv_len"], s["page_table"], s["free"], s["count"], page_size=c["page"], total_q=s["total"],
                  keep_len=s["keep"], shared_pages=c["shared"], kv_len_out=s["kv_out"], free_count_out=s["count_out"],
                  q_start=s["q_start"], slots=s["slots"], positions=s["positions"])
    return s["kv_out"], s["count_out"], s["q_start"], s["page_table"], s["free"], s["slots"], s["positions"]


def _append_own(s):
    from block_sparse_attention_fa_gb300 import fa
    fa.kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], s["q_start"],
                 k_scale=s["k_scale"], v_scale=s["v_scale"], cos=s["cos"], sin=s["sin"],
                 interleaved=s["case"]["interleaved"], q_out=s["q_out"])
    return s["q_out"], s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]


def _paged_own(s):
    from block_sparse_attention_fa_gb300 import fa
    c = s["case"]
    return fa.fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], s["q_start"],
                        k_scale=s["k_scale"], v_scale=s["v_scale"], max_q_len=s["max_q"],
                        mask="causal" if c["window"] < 0 else "sink_window", window=max(c["window"], 0),
                        sinks=c["sinks"] if c["window"] >= 0 else 0, shared_len=c["shared"],
                        score="softcap" if c["cap"] else "none", softcap=c["cap"])


def _step_plain(s):
    c = s["case"]
    P, S, B = c["page"], c["shared"], c["B"]
    old, keep, new, table, free = s["kv_len"].long(), s["keep"].long(), s["new"].long(), s["page_table"], s["free"]
    F, width, cap = s["count"].long(), s["page_table"].shape[1], s["free"].numel()
    length = keep + new
    before, after = ((old + P - 1) // P).clamp(min=S), ((length + P - 1) // P).clamp(min=S)
    take, give = (after - before).clamp(min=0), (before - after).clamp(min=0)
    R, N = give.sum(), take.sum()
    # pages given back, on top of the stack, the last request's last page first
    e = torch.arange(width, device=DEVICE)[None]
    gone = (e >= after[:, None]) & (e < before[:, None])
    r = F + R - 1 - ((give.cumsum(0) - give)[:, None] + e - after[:, None])
    stack = torch.cat([free, free[:1]])
    stack[torch.where(gone, r, torch.full_like(r, cap))] = table
    free.copy_(stack[:cap])
    # pages taken, from the top
    come = (e >= before[:, None]) & (e < after[:, None])
    k = F + R - 1 - ((take.cumsum(0) - take)[:, None] + e - before[:, None])
    table.copy_(torch.where(come, free[k.clamp(0, cap - 1)], table))
    ends = new.cumsum(0)
    s["kv_out"].copy_(length)
    s["count_out"].copy_(F + R - N)
    s["q_start"][1:] = ends
    s["q_start"][0] = 0
    row = torch.arange(s["total"], device=DEVICE)
    b = torch.searchsorted(ends, row, right=True)
    here = b < B
    b = b.clamp(max=B - 1)
    pos = keep[b] + row - (ends - new)[b]
    slot = table[b, (pos // P).clamp(max=width - 1)].long() * P + pos % P
    s["slots"].copy_(torch.where(here, slot, torch.full_like(slot, -1)))
    s["positions"].copy_(torch.where(here, pos, torch.zeros_like(pos)))
    return s["kv_out"], s["count_out"], s["q_start"], s["page_table"], s["free"], s["slots"], s["positions"]


def _tokens(s):
    """Sequence and position of every row that belongs to one."""
    row = torch.arange(s["rows"], device=DEVICE)
    start = s["q_start"].long()
    b = torch.searchsorted(start[1:], row, right=True)
    return row, b, s["kv_len"].long()[b] - (start[b + 1] - row)


def _rotate(x, cos, sin, interleaved):
    half = cos.shape[-1]
    a, rest = x.float()[..., : 2 * half], x.float()[..., 2 * half:]
    if interleaved:
        x0, x1 = a[..., 0::2], a[..., 1::2]
        a = torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2)
    else:
        x0, x1 = a[..., :half], a[..., half:]
        a = torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1)
    return torch.cat([a, rest], -1)


def _to_e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _put8(s, name, x, b, pos):
    """Rows x [rows, Hkv, D] (32 bits) into the cache `name`."""
    P = s["case"]["page"]
    cache, scale = s[name + "_cache"].view(torch.uint8), s[name + "_scale"]
    table = s["page_table"].long()
    page, slot = table[b, pos // P], pos % P
    amax = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand(x.shape[:2]), x.abs().amax(-1), "amax")
    # the page of each sequence's first new token may hold earlier ones
    start = s["q_start"].long()
    at = s["kv_len"].long() - (start[1:] - start[:-1])
    first, earlier = table[torch.arange(len(at), device=DEVICE), at // P], at % P
    before = scale[first]
    need = _pow2_scale(amax)
    after = torch.where(earlier[:, None] > 0, torch.maximum(before, need[first]), need[first])
    written = torch.zeros(scale.shape[0], dtype=torch.bool, device=DEVICE)
    written[page] = True
    scale.copy_(torch.where(written[:, None], need, scale))
    scale[first] = after
    old = cache[first]
    turned = _to_e4m3(old.view(torch.float8_e4m3fn).float() * (before / after)[:, :, None, None])
    keep = torch.arange(P, device=DEVICE)[None] < earlier[:, None]
    cache[first] = torch.where(keep[:, None, :, None], turned, old)
    cache[page, :, slot] = _to_e4m3(x / scale[page][:, :, None])


def _append_plain(s):
    c, n = s["case"], s["rows"]
    row, b, pos = _tokens(s)
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    s["q_out"][:n] = _rotate(s["q"][:n], cos, sin, c["interleaved"]).to(torch.bfloat16)
    _put8(s, "k", _rotate(s["k"][:n], cos, sin, c["interleaved"]), b, pos)
    _put8(s, "v", s["v"][:n].float(), b, pos)
    return s["q_out"], s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]


def _seen(i, j, window, sinks):
    see = j <= i
    return see if window < 0 else see & ((i - j <= window) | (j < sinks))


def _values(s, name, page, slot):
    """What the cache holds of these pages and slots, in 32 bits: [..., Hkv, D]."""
    codes = s[name + "_cache"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn)
    return codes.float() * s[name + "_scale"][page][..., None]


def _paged_plain(s):
    c = s["case"]
    B, Hkv, P, D, shared = c["B"], c["Hkv"], c["page"], c["D"], c["shared"]
    group, n = c["Hq"] // Hkv, s["max_q"]
    row, b, pos = _tokens(s)
    turn = row - s["q_start"].long()[b]
    # the sequences' own keys, padded to the longest; the prefix once
    j = shared + torch.arange(s["longest"], device=DEVICE)
    page = s["page_table"].long()[:, (j // P).clamp(max=s["page_table"].shape[1] - 1)].clamp(min=0)
    slot = (j % P)[None].expand_as(page)
    k = _values(s, "k", page, slot).permute(0, 2, 1, 3)
    v = _values(s, "v", page, slot).permute(0, 2, 1, 3)
    q = torch.zeros((B, n, Hkv, group, D), device=DEVICE)
    q[b, turn] = s["q"].float().view(-1, Hkv, group, D)
    i = torch.zeros((B, n), dtype=torch.long, device=DEVICE)
    i[b, turn] = pos
    q = q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, group * n, D) / math.sqrt(D)
    i = i[:, None, :].expand(B, group, n).reshape(B, 1, group * n, 1)

    def scores(keys, at):
        x = q @ keys.transpose(-1, -2)
        if c["cap"]:
            x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
        return x.masked_fill_(~_seen(i, at, c["window"], c["sinks"]), -math.inf)

    x = scores(k, j)
    if shared:
        j0 = torch.arange(shared, device=DEVICE)
        p0 = s["page_table"].long()[0, j0 // P]
        k0, v0 = (_values(s, name, p0, j0 % P).transpose(0, 1) for name in "kv")
        x = torch.cat([scores(k0, j0), x], -1)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = p[..., shared:] @ v
    if shared:
        o = o + p[..., :shared] @ v0
    o = (o / total).view(B, Hkv, group, n, D).permute(0, 3, 1, 2, 4)[b, turn]
    lse = (m + total.log()).view(B, Hkv, group, n).permute(0, 3, 1, 2)[b, turn]
    return o.reshape(-1, c["Hq"], D).to(s["q"].dtype), lse.reshape(-1, c["Hq"])


# -------------------------------------------------------------------- work
def _pairs(lo, hi, window, sinks):
    """Visible (query, key) pairs of queries at positions lo .. hi - 1 (keys from 0)."""
    i = np.arange(lo, hi, dtype=np.float64)
    if window < 0:
        return float((i + 1).sum())
    first = np.maximum(i - window, 0)
    return float((i + 1 - first + np.minimum(first, sinks)).sum())


def work(case):
    if case["op"] == "step":
        old, keep, new = _requests(case)
        before, after = _page_counts(case, old, keep, new)
        moved = int(np.abs(after - before).sum())
        rows = int(new.sum()) + case["pad"]
        # three lengths in, one and the offset out; page ids moved; slot and position of every row
        return {"bytes": 20 * case["B"] + 8 * moved + 12 * rows, "flops": 10 * rows}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    new, kv = _lengths(case)
    rows = int(new.sum())
    if case["op"] == "append":
        return {"bytes": rows * ((4 * Hq + 6 * Hkv) * D + 4 * case["rot"]),
                "flops": rows * (3 * (Hq + Hkv) * case["rot"] + 4 * Hkv * D)}
    shared, window, sinks = case["shared"], case["window"], case["sinks"]
    pairs = sum(_pairs(shared + L - n, shared + L, window, sinks) for n, L in zip(new.tolist(), kv.tolist()))
    # the keys that some query of the sequence sees, the prefix's once for the batch
    total, front = 0, 0
    for n, L in zip(new.tolist(), kv.tolist()):
        first = 0 if window < 0 else max(0, shared + L - n - window)
        total += shared + L - max(first, shared) + max(0, min(sinks, first) - shared)
        front = max(front, shared - min(first, shared) + min(sinks, first, shared))
    return {"bytes": 2 * Hkv * D * (total + front) + rows * Hq * (4 * D + 4), "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------- exact
def _step_exact(s):
    """The definition, request by request."""
    c = s["case"]
    P, S = c["page"], c["shared"]
    table, free = s["page_table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    top = int(s["count"][0])
    old, keep, new = (s[x].cpu().numpy() for x in ("kv_len", "keep", "new"))
    had = [max(-(-int(x) // P), S) for x in old]
    has = [max(-(-int(x) // P), S) for x in keep + new]
    for b in reversed(range(c["B"])):
        for e in reversed(range(has[b], had[b])):
            free[top] = table[b, e]
            top += 1
    start, slots, places = [0], np.full(s["total"], -1, np.int64), np.zeros(s["total"], np.int32)
    for b in range(c["B"]):
        for e in range(had[b], has[b]):
            top -= 1
            table[b, e] = free[top]
        at = keep[b] + np.arange(new[b])
        rows = slice(start[-1], start[-1] + new[b])
        slots[rows] = table[b, at // P].astype(np.int64) * P + at % P
        places[rows] = at
        start.append(start[-1] + int(new[b]))
    return (keep + new).astype(np.int32), np.array([top], np.int32), np.array(start, np.int32), table, free, slots, places


def _e4m3_64(y):
    """The e4m3 number nearest to each y (ties to even), in 64 bits."""
    a = y.abs().clamp(max=E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign(torch.round(a / step) * step, y).clamp(-E4M3_MAX, E4M3_MAX)


def _append_exact(s):
    c = s["case"]
    P = c["page"]
    start, lens, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["page_table"].cpu()
    q_out = s["q_out"].double()
    caches = {n: s[n + "_cache"].double() for n in "kv"}
    scales = {n: s[n + "_scale"].double() for n in "kv"}
    half = c["rot"] // 2
    one = torch.arange(half, device=DEVICE) * (2 if c["interleaved"] else 1)
    two = one + (1 if c["interleaved"] else half)
    # the tables hold 32 bits: they are inputs, and taken as they are
    cos, sin = s["cos"].double(), s["sin"].double()

    def turned(x, at):
        y = x.double().clone()
        a, b = x.double()[..., one], x.double()[..., two]
        y[..., one] = a * cos[at][:, None] - b * sin[at][:, None]
        y[..., two] = b * cos[at][:, None] + a * sin[at][:, None]
        return y

    for b, L in enumerate(lens):
        lo, hi = start[b], start[b + 1]
        n = hi - lo
        at = torch.arange(L - n, L, device=DEVICE)
        q_out[lo:hi] = turned(s["q"][lo:hi], at)
        rows = dict(k=turned(s["k"][lo:hi], at), v=s["v"][lo:hi].double())
        for e in range((L - n) // P, (L - 1) // P + 1):
            page, f, t = int(table[b, e]), max(e * P, L - n), min((e + 1) * P, L)
            for name in "kv":
                x = rows[name][f - (L - n): t - (L - n)]                     # [tokens, Hkv, D]
                # the smallest power of two s with amax <= 448 s, without logarithms: count the ones that are too small
                powers = torch.exp2(torch.arange(*SCALE_EXP, device=DEVICE, dtype=torch.float64))
                few = (x.abs().amax((0, 2))[:, None] > E4M3_MAX * powers[None]).sum(1)
                scale = torch.exp2((few + SCALE_EXP[0]).double())
                if f > e * P:
                    scale = torch.maximum(scale, scales[name][page])
                    codes = caches[name][page, :, : f - e * P]
                    caches[name][page, :, : f - e * P] = _e4m3_64(codes * (scales[name][page] / scale)[:, None, None])
                scales[name][page] = scale
                caches[name][page, :, f - e * P: t - e * P] = _e4m3_64(x.transpose(0, 1) / scale[:, None, None])
    return q_out, caches["k"], scales["k"], caches["v"], scales["v"]


def _paged_exact(s):
    c = s["case"]
    D, group = c["D"], c["Hq"] // c["Hkv"]
    start, lens, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["page_table"].long()
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEVICE)
    codes = {n: s[n + "_cache"].view(torch.uint8) for n in "kv"}
    for b, L in enumerate(lens):
        lo, n = start[b], start[b + 1] - start[b]
        pages = table[b, : -(-L // c["page"])]
        j = torch.arange(L, device=DEVICE)
        far = torch.arange(L - n, L, device=DEVICE)[:, None] - j[None]
        see = far >= 0
        if c["window"] >= 0:
            see &= (far <= c["window"]) | (j[None] < c["sinks"])
        see = see.repeat(group, 1)
        for h in range(c["Hkv"]):
            k, v = ((codes[name][pages, h].view(torch.float8_e4m3fn).double()
                     * s[name + "_scale"][pages, h].double()[:, None, None]).reshape(-1, D)[:L] for name in "kv")
            q = s["q"][lo: lo + n, h * group: (h + 1) * group].transpose(0, 1).reshape(-1, D).double()
            x = q @ k.T / math.sqrt(D)
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            x = torch.where(see, x, torch.full_like(x, -math.inf))
            y = torch.logsumexp(x, -1)
            o[lo: lo + n, h * group: (h + 1) * group] = (torch.exp(x - y[:, None]) @ v).view(group, n, -1).transpose(0, 1)
            lse[lo: lo + n, h * group: (h + 1) * group] = y.view(group, n).T
    return o, lse


def exact(case, seed):
    w = work(case)
    if w["flops"] > 4e12:
        return None
    return {"step": _step_exact, "append": _append_exact, "paged": _paged_exact}[case["op"]](prepare(case, seed))
