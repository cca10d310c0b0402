"""Cases, plain forms and exact values of the serving and sink-window operators.

Four operators, in the framework's order of use: attention under a sliding
window with sink tokens (forward and backward), appending rotated keys and
values to a paged cache, attention over the paged cache, and the same for a
batch whose sequences share a long prefix.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
ROPE_BASE = 10000.0


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a training step of one layer: 32 query heads on 8 kv heads, 8192 tokens
        dict(name="sink_train_8k", op="sinks", dtype="bf16", B=1, Hq=32, Hkv=8, T=8192, D=128, window=1024, sinks=4),
        # a short odd batch with one kv head per query head and more sinks than a tile holds
        dict(name="sink_train_odd", op="sinks", dtype="bf16", B=2, Hq=8, Hkv=8, T=1531, D=64, window=200, sinks=130),
        # exact fp32 scoring of a few grouped windows (forward only)
        dict(name="sink_fp32", op="sinks", dtype="fp32", B=1, Hq=4, Hkv=4, T=136, D=128, window=32, sinks=4),
        # one decoding step of 64 sequences
        dict(name="append_step", op="append", B=64, q_len=1, kv_len=1024, Hq=32, Hkv=8, D=128, page=16, rot=128,
             interleaved=False, ragged=True, pad=0),
        # ragged prompts, interleaved pairs, half of the head rotated, rows of padding behind the last prompt
        dict(name="append_prompts", op="append", B=8, q_len=4096, kv_len=4096, Hq=32, Hkv=8, D=128, page=64, rot=64,
             interleaved=True, ragged=True, pad=37),
        # one user, a short context: latency
        dict(name="paged_one", op="paged", B=1, q_len=1, kv_len=520, Hq=32, Hkv=8, D=128, page=16, window=-1, sinks=0,
             ragged=False, shared=0),
        # long contexts of equal length, one token each
        dict(name="paged_long", op="paged", B=8, q_len=1, kv_len=32768, Hq=32, Hkv=8, D=128, page=64, window=-1,
             sinks=0, ragged=False, shared=0),
        # streaming: ragged contexts, 3 tokens to verify each, window and sinks
        dict(name="paged_stream", op="paged", B=64, q_len=3, kv_len=16384, Hq=16, Hkv=4, D=64, page=16, window=1024,
             sinks=4, ragged=True, shared=0),
        # the second chunk of long prompts
        dict(name="paged_chunk", op="paged", B=4, q_len=1024, kv_len=8192, Hq=32, Hkv=8, D=128, page=128, window=-1,
             sinks=0, ragged=True, shared=0),
        # 64 chats over one long system prompt, one token each
        dict(name="shared_chat", op="paged", B=64, q_len=1, kv_len=512, Hq=32, Hkv=8, D=128, page=64, window=-1,
             sinks=0, ragged=True, shared=16384),
        # 16 candidates of 4 tokens each after one document; the prefix ends inside a tile
        dict(name="shared_verify", op="paged", B=16, q_len=4, kv_len=200, Hq=16, Hkv=4, D=64, page=32, window=-1,
             sinks=0, ragged=True, shared=5024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sinks", "append", "paged", "paged", "shared"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    window = rng.choice([-1, -1, _log_int(rng, 1, 4096)])
    sinks = rng.choice([0, 1, 4, _log_int(rng, 1, 300)])
    if op == "sinks":
        if rng.random() < 0.25:
            return dict(op="sinks", dtype="fp32", B=rng.randint(1, 3), Hq=2 * group, Hkv=2, T=_log_int(rng, 1, 700), D=D,
                        window=_log_int(rng, 1, 300), sinks=sinks)
        T = _log_int(rng, 1, 6000)
        return dict(op="sinks", dtype="bf16", B=rng.randint(1, 2), Hq=2 * group, Hkv=2, T=T, D=D,
                    window=_log_int(rng, 1, 2048), sinks=sinks)
    if op == "append":
        n = _log_int(rng, 1, 2000)
        return dict(op="append", B=_log_int(rng, 1, max(2, min(128, 16000 // n))), q_len=n,
                    kv_len=n + _log_int(rng, 1, 2000), Hq=Hkv * group, Hkv=Hkv, D=D, page=page,
                    rot=rng.choice([32, 64, D]), interleaved=rng.random() < 0.5, ragged=rng.random() < 0.7,
                    pad=rng.randint(0, 9))
    if op == "shared":
        n = rng.choice([1, 1, 2, 4, 7])
        return dict(op="paged", B=_log_int(rng, 2, 64), q_len=n, kv_len=n + _log_int(rng, 1, 700), Hq=Hkv * group,
                    Hkv=Hkv, D=D, page=page, window=window, sinks=sinks, ragged=True,
                    shared=page * rng.randint(1, max(1, _log_int(rng, 300, 16000) // page)))
    n = rng.choice([1, 1, 2, 5, _log_int(rng, 1, 1000)])
    kv = n + _log_int(rng, 1, 30000 if n < 8 else 6000)
    most = max(1, min(64, 250000 // kv, 80000 // (n * Hkv * group)))
    return dict(op="paged", B=_log_int(rng, 1, most), q_len=n, kv_len=kv,
                Hq=Hkv * group, Hkv=Hkv, D=D, page=page, window=window, sinks=sinks, ragged=rng.random() < 0.7, shared=0)


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dtype)


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
    B, page, shared = case["B"], case["page"], case.get("shared", 0)
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


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "sinks":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        B, T = case["B"], case["T"]
        s = dict(q=_normal(gen, (B, Hq, T, D), dt), k=_normal(gen, (B, Hkv, T, D), dt), v=_normal(gen, (B, Hkv, T, D), dt))
        if case["dtype"] == "bf16":
            s["dout"] = _normal(gen, (B, Hq, T, D), dt)
        return dict(case=case, **s)
    new, kv = _lengths(case)
    s = dict(case=case, **_pages(case, new, kv, gen), max_q=case["q_len"])
    cache = (s["num_pages"], Hkv, case["page"], D)
    s["k_cache"], s["v_cache"] = _normal(gen, cache), _normal(gen, cache)
    if case["op"] == "append":
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
    s["q"] = _normal(gen, (s["rows"], Hq, D))
    return s


# --------------------------------------------------------------- operators
def run(state):
    case = state["case"]
    if case["op"] == "sinks":
        return _sinks_own(state) if own else _sinks_plain(state)
    if case["op"] == "append":
        return _append_own(state) if own else _append_plain(state)
    return _paged_own(state) if own else _paged_plain(state)


def _sinks_own(s):
    from block_sparse_attention_fa_gb300 import fa
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    bm = fa.block_mask("sink_window", 1, 1, c["T"], c["T"], window=c["window"], sinks=c["sinks"], device=q.device)
    o, lse = fa.fwd(q, k, v, bm)
    if "dout" not in s:
        return o, lse
    dq, dk, dv = fa.bwd(q, k, v, o, lse, s["dout"], bm)
    # the parameters are bf16, and so are the gradients that reach them
    return o, lse, dq.to(q.dtype), dk.to(q.dtype), dv.to(q.dtype)


def _append_own(s):
    from block_sparse_attention_fa_gb300 import fa
    fa.kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], s["q_start"],
                 cos=s["cos"], sin=s["sin"], interleaved=s["case"]["interleaved"], q_out=s["q_out"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _paged_own(s):
    from block_sparse_attention_fa_gb300 import fa
    c = s["case"]
    mask = "causal" if c["window"] < 0 else "sink_window"
    return fa.fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], s["q_start"],
                        max_q_len=s["max_q"], mask=mask, window=max(c["window"], 0),
                        sinks=c["sinks"] if c["window"] >= 0 else 0, shared_len=c["shared"])


def _seen(i, j, window, sinks):
    see = j <= i
    return see if window < 0 else see & ((i - j <= window) | (j < sinks))


def _sinks_plain(s):
    c, dt = s["case"], s["q"].dtype
    B, Hq, T, D = s["q"].shape
    Hkv = s["k"].shape[1]
    scale = 1.0 / math.sqrt(D)
    q = s["q"].float().view(B, Hkv, Hq // Hkv, T, D)
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    at = torch.arange(T, device=q.device)
    hidden = ~_seen(at[:, None], at[None], c["window"], c["sinks"])
    x = (q @ k.transpose(-1, -2) * scale).masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(total)
    o = p @ v
    lse = (m + total.log()).view(B, Hq, T)
    if "dout" not in s:
        return o.view(B, Hq, T, D).to(dt), lse
    do = s["dout"].float().view_as(q)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = do @ v.transpose(-1, -2)
    ds = ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = ds @ k
    dk = (ds.transpose(-1, -2) @ q).sum(2)
    return o.view(B, Hq, T, D).to(dt), lse, dq.view(B, Hq, T, D).to(dt), dk.to(dt), dv.to(dt)


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
    return torch.cat([a, rest], -1).to(x.dtype)


def _append_plain(s):
    c, n = s["case"], s["rows"]
    row, b, pos = _tokens(s)
    page, slot = s["page_table"].long()[b, pos // c["page"]], pos % c["page"]
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    s["q_out"][:n] = _rotate(s["q"][:n], cos, sin, c["interleaved"])
    s["k_cache"][page, :, slot] = _rotate(s["k"][:n], cos, sin, c["interleaved"])
    s["v_cache"][page, :, slot] = s["v"][:n]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _paged_plain(s):
    c = s["case"]
    B, Hkv, page, D, shared = c["B"], c["Hkv"], c["page"], c["D"], c["shared"]
    group, n = c["Hq"] // Hkv, s["max_q"]
    row, b, pos = _tokens(s)
    turn = row - s["q_start"].long()[b]
    # the sequences' own keys, padded to the longest; the prefix once
    j = shared + torch.arange(s["longest"], device=DEVICE)
    own_page = s["page_table"].long()[:, (j // page).clamp(max=s["page_table"].shape[1] - 1)].clamp(min=0)
    k = s["k_cache"][own_page, :, j % page].float().permute(0, 2, 1, 3)
    v = s["v_cache"][own_page, :, j % page].float().permute(0, 2, 1, 3)
    q = torch.zeros((B, n, Hkv, group, D), device=DEVICE)
    q[b, turn] = s["q"].float().view(-1, Hkv, group, D)
    i = torch.zeros((B, n), dtype=torch.long, device=DEVICE)
    i[b, turn] = pos
    q = q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, group * n, D) / math.sqrt(D)
    i = i[:, None, :].expand(B, group, n).reshape(B, 1, group * n, 1)
    x = (q @ k.transpose(-1, -2)).masked_fill_(~_seen(i, j, c["window"], c["sinks"]), -math.inf)
    if shared:
        j0 = torch.arange(shared, device=DEVICE)
        p0 = s["page_table"].long()[0, j0 // page]
        k0 = s["k_cache"][p0, :, j0 % page].float().transpose(0, 1)
        v0 = s["v_cache"][p0, :, j0 % page].float().transpose(0, 1)
        x0 = (q @ k0.transpose(-1, -2)).masked_fill_(~_seen(i, j0, c["window"], c["sinks"]), -math.inf)
        x = torch.cat([x0, x], -1)
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
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "sinks":
        B, T = case["B"], case["T"]
        pairs = B * Hq * _pairs(0, T, case["window"], case["sinks"])
        qo, kv, e = B * Hq * T * D, B * Hkv * T * D, 2 if case["dtype"] == "bf16" else 4
        if case["dtype"] == "fp32":
            return {"bytes": e * (2 * qo + 2 * kv) + 4 * B * Hq * T, "flops": 4 * D * pairs}
        # q, k, v, dout in; o, lse and the three gradients out
        return {"bytes": e * (4 * qo + 4 * kv) + 4 * B * Hq * T, "flops": 14 * D * pairs}
    new, kv = _lengths(case)
    rows = int(new.sum())
    if case["op"] == "append":
        return {"bytes": rows * (4 * (Hq + 2 * Hkv) * D + 4 * case["rot"]), "flops": 3 * rows * (Hq + Hkv) * case["rot"]}
    shared, window, sinks = case["shared"], case["window"], case["sinks"]
    pairs = sum(_pairs(shared + L - n, shared + L, window, sinks) for n, L in zip(new.tolist(), kv.tolist()))
    # the keys that some query of the sequence sees, the prefix's once for the batch
    total, front = 0, 0
    for n, L in zip(new.tolist(), kv.tolist()):
        first = 0 if window < 0 else max(0, shared + L - n - window)
        total += shared + L - max(first, shared) + max(0, min(sinks, first) - shared)
        front = max(front, shared - min(first, shared) + min(sinks, first, shared))
    return {"bytes": 4 * Hkv * D * (total + front) + rows * Hq * (4 * D + 4), "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------- exact
def _attend64(q, k, v, see):
    """Rows of q against k, v in 64 bits, one head: (o, lse); `see` is the visibility of every pair."""
    x = torch.where(see, (q.double() @ k.double().T) / math.sqrt(q.shape[-1]), torch.tensor(-math.inf, dtype=torch.float64, device=q.device))
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - lse[:, None])
    return w @ v.double(), lse, w


def _sinks_exact(s):
    c = s["case"]
    B, Hq, T, D = s["q"].shape
    Hkv = s["k"].shape[1]
    i = torch.arange(T, device=DEVICE)
    far = i[:, None] - i[None]
    see = (far >= 0) & ((far <= c["window"]) | (i[None] < c["sinks"]))
    o, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE), torch.zeros((B, Hq, T), dtype=torch.float64, device=DEVICE)
    dq, dk, dv = torch.zeros_like(o), torch.zeros(s["k"].shape, dtype=torch.float64, device=DEVICE), torch.zeros(s["k"].shape, dtype=torch.float64, device=DEVICE)
    for b in range(B):
        for h in range(Hq):
            g = h * Hkv // Hq
            q, k, v = s["q"][b, h].double(), s["k"][b, g].double(), s["v"][b, g].double()
            o[b, h], lse[b, h], w = _attend64(q, k, v, see)
            if "dout" in s:
                do = s["dout"][b, h].double()
                dw = w * (do @ v.T - (do * o[b, h]).sum(-1)[:, None]) / math.sqrt(D)
                dq[b, h] = dw @ k
                dk[b, g] += dw.T @ q
                dv[b, g] += w.T @ do
    return (o, lse, dq, dk, dv) if "dout" in s else (o, lse)


def _append_exact(s):
    c = s["case"]
    start, lens, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["page_table"].cpu()
    q_out, kc, vc = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
    half = c["rot"] // 2
    if c["interleaved"]:
        one = torch.arange(half, device=DEVICE) * 2
        two = one + 1
    else:
        one = torch.arange(half, device=DEVICE)
        two = one + half
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
        at = torch.arange(L - (hi - lo), L)
        pages, slots = table[b, at // c["page"]].long().to(DEVICE), (at % c["page"]).to(DEVICE)
        at = at.to(DEVICE)
        q_out[lo:hi] = turned(s["q"][lo:hi], at)
        kc[pages, :, slots] = turned(s["k"][lo:hi], at)
        vc[pages, :, slots] = s["v"][lo:hi].double()
    return q_out, kc, vc


def _paged_exact(s):
    c = s["case"]
    start, lens, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["page_table"].long()
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEVICE)
    group = c["Hq"] // c["Hkv"]
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
            k = s["k_cache"][pages, h].reshape(-1, c["D"])[:L]
            v = s["v_cache"][pages, h].reshape(-1, c["D"])[:L]
            q = s["q"][lo: lo + n, h * group: (h + 1) * group].transpose(0, 1).reshape(-1, c["D"])
            x, y, _ = _attend64(q, k, v, see)
            o[lo: lo + n, h * group: (h + 1) * group] = x.view(group, n, -1).transpose(0, 1)
            lse[lo: lo + n, h * group: (h + 1) * group] = y.view(group, n).T
    return o, lse


def exact(case, seed):
    w = work(case)
    if w["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    return {"sinks": _sinks_exact, "append": _append_exact, "paged": _paged_exact}[case["op"]](s)
