"""Measured cases of the paged key/value cache operators.

The operators: the page map (block tables and slot maps from request lengths),
the append of new tokens to the pages, the pages' key bounds, the selection of
pages by a score on those bounds, and the attention of one new token per
sequence over the pages.  Every case of `listed()` is one call; `run` computes
it from elementary torch operations, or with `own` through global_gqa_b200.

Head shapes are those of Gemma 3 27B (32 query / 16 kv heads of 128), 1B (4 / 1
heads of 256) and of this repository's tests; lengths are those of its decode
workload (contexts of 4K to 128K tokens).
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
NEG = float("-inf")


def _g3():
    import global_gqa_b200
    return global_gqa_b200


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One serving step of 64 running requests: one new token each.
        dict(name="map_step_b64", op="map", B=64, old_lo=4096, old_hi=131071, new_lo=1, new_hi=1, idle=0, P=64,
             max_pages=2048, short=False),
        # Admission of ragged prompts beside requests that wait (no new token).
        dict(name="map_prompts_b1024", op="map", B=1024, old_lo=0, old_hi=4096, new_lo=1, new_hi=500, idle=100, P=16,
             max_pages=512, short=False),
        # The new tokens of 64 running requests, 27B heads, a global layer.
        dict(name="append_step_b64", op="append", T=64, pad=0, Hq=32, Hkv=16, D=128, P=64, base=1e6, interp=8.0, hi=131072),
        # A packed 8K prompt batch with some padding rows behind it.
        dict(name="append_prompt_8k", op="append", T=8192, pad=150, Hq=32, Hkv=16, D=128, P=64, base=1e6, interp=8.0,
             hi=32768),
        # After a decode step: the last page of each of 64 sequences.
        dict(name="bounds_step_b64", op="bounds", B=64, lo=4096, hi=16384, step=True, Hkv=16, D=128, P=64),
        # After prompts of up to 32K tokens: all their pages.
        dict(name="bounds_prompts_b8", op="bounds", B=8, lo=4096, hi=32768, step=False, Hkv=16, D=128, P=64),
        # One 1B-shaped sequence of 32K tokens in small pages.
        dict(name="select_b1_32k", op="select", B=1, lo=32768, hi=32768, Hq=4, Hkv=1, D=256, P=16, n_select=64),
        # The batched decode workload: 64 sequences of 4K to 128K tokens.
        dict(name="select_b64_128k", op="select", B=64, lo=4096, hi=131072, Hq=32, Hkv=16, D=128, P=64, n_select=64),
        # One interactive user at 4K tokens: latency.
        dict(name="decode_b1_4k", op="decode", B=1, lo=4096, hi=4096, Hq=32, Hkv=16, D=128, P=64, window=0, n_select=0),
        # A global layer of a full batch.
        dict(name="decode_b64_32k", op="decode", B=64, lo=4096, hi=32768, Hq=32, Hkv=16, D=128, P=64, window=0,
             n_select=0),
        # A sliding-window layer of the same batch; pages before the window were given back.
        dict(name="decode_local_b64", op="decode", B=64, lo=4096, hi=131072, Hq=32, Hkv=16, D=128, P=64, window=1024,
             n_select=0),
        # Sparse decode: 32 selected pages of each sequence and kv head.
        dict(name="decode_selected_b32", op="decode", B=32, lo=8192, hi=65536, Hq=32, Hkv=16, D=128, P=64, window=0,
             n_select=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["map", "append", "bounds", "select", "decode", "decode"])
    P = rng.choice([16, 32, 64, 128])
    Hkv, G, D = rng.choice([(16, 2, 128), (1, 4, 256), (2, 2, 64), (2, 4, 128), (4, 1, 128), (1, 4, 64), (8, 3, 128),
                            (2, 8, 128), (3, 5, 64)])
    if op == "map":
        B, new_hi = _log(rng, 2, 1024), _log(rng, 4, 500)
        old_hi = _log(rng, 100, 8000)
        return dict(op=op, B=B, old_lo=0, old_hi=old_hi, new_lo=0, new_hi=new_hi, idle=rng.randint(0, B // 4), P=P,
                    max_pages=(old_hi + new_hi + P - 1) // P + rng.randint(0, 9), short=rng.random() < 0.3)
    if op == "append":
        T = _log(rng, 1, 8192 * 16 // max(Hkv, 16))
        return dict(op=op, T=T, pad=rng.randint(0, T // 8), Hq=Hkv * G, Hkv=Hkv, D=D, P=P, base=rng.choice([1e4, 1e6]),
                    interp=rng.choice([1.0, 8.0]), hi=_log(rng, T + 1, 131072))
    if op == "bounds":
        B, hi = _log(rng, 1, 16), _log(rng, 1, 16384)
        return dict(op=op, B=B, lo=_log(rng, 1, hi), hi=hi, step=rng.random() < 0.3, Hkv=Hkv, D=D, P=P)
    hi = _log(rng, 1, 32768) if op == "decode" else _log(rng, 32 * P, 65536)
    B = _log(rng, 1, max(1, min(64, 16 * 32768 * 16 * 128 // (hi * Hkv * D))))
    if op == "select":  # some sequences have fewer pages than are selected
        return dict(op=op, B=B, lo=_log(rng, 1, hi), hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, P=P,
                    n_select=_log(rng, 3, min(200, hi // P // 2)))
    kind = rng.choice(["all", "all", "window", "selected"])
    return dict(op=op, B=B, lo=_log(rng, 1, hi), hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, P=P,
                window=_log(rng, 1, 1024) if kind == "window" else 0, n_select=_log(rng, 1, 64) if kind == "selected" else 0)


# ------------------------------------------------------------------ inputs
class _Gen:
    """Random numbers of one seed: small integers from the CPU, large tensors on the GPU."""

    def __init__(self, seed):
        self.c = torch.Generator().manual_seed(seed)
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def ints(self, lo, hi, n):
        return torch.randint(lo, hi + 1, (n,), generator=self.c)

    def normal(self, *shape, dtype=torch.bfloat16):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        flat = out.view(-1)
        for s in range(0, flat.numel(), 1 << 28):  # bounds the fp32 temporary of a large pool
            n = min(1 << 28, flat.numel() - s)
            flat[s:s + n] = torch.randn(n, generator=self.g, device="cuda").to(dtype)
        return out

    def gain(self, D):
        return 1.0 + 0.1 * torch.randn(D, generator=self.g, device="cuda")


def _lengths(c, r):
    """Sequence lengths in [lo, hi]; the first is hi, so that a case's work hardly depends on the seed."""
    L = r.ints(c["lo"], c["hi"], c["B"])
    L[0] = c["hi"]
    return L


def _table(r, counts, first, max_pages):
    """Block table [B, max_pages] of pages scattered over a pool: entries first[b] .. first[b]+counts[b]-1, -1 elsewhere."""
    total = int(counts.sum())
    perm = torch.randperm(total, generator=r.c).to(torch.int32)
    t = torch.full((len(counts), max_pages), -1, dtype=torch.int32)
    col = torch.arange(max_pages)
    t[(col >= first[:, None]) & (col < (first + counts)[:, None])] = perm
    return t.cuda(), total


def prepare(case, seed):
    c, r = case, _Gen(seed)
    i32 = lambda t: t.to(torch.int32).cuda()  # noqa: E731
    if c["op"] == "map":
        old, new = r.ints(c["old_lo"], c["old_hi"], c["B"]), r.ints(c["new_lo"], c["new_hi"], c["B"])
        new[torch.randperm(c["B"], generator=r.c)[:c["idle"]]] = 0
        have = (old + c["P"] - 1) // c["P"]
        table, used = _table(r, have, torch.zeros_like(have), c["max_pages"])
        need = int(((old + new + c["P"] - 1) // c["P"] - have).sum())
        n_free = need * 2 // 3 if c["short"] else need + 17
        n_pages = used + n_free + 5
        ring = torch.full((n_pages,), -1, dtype=torch.int32)  # the free ring: n_free live entries, wrapping round its end
        head = n_pages - n_free // 3 - 1
        ring[(head + torch.arange(n_free)) % n_pages] = (used + torch.randperm(n_free, generator=r.c)).to(torch.int32)
        return dict(op="map", P=c["P"], n_pages=n_pages, max_tokens=c["B"] * c["new_hi"] + 13, old=i32(old), new=i32(new),
                    table=table, ring=ring.cuda(), ring_state=i32(torch.tensor([head, n_free])))
    if c["op"] == "append":
        T, Hq, Hkv, D, P = c["T"], c["Hq"], c["Hkv"], c["D"], c["P"]
        n_pages = T // P + 9
        slots = torch.randperm(n_pages * P, generator=r.c)[:T]
        slots[T - c["pad"]:] = -1
        pos = r.ints(0, c["hi"] - 1, T)
        pos[T - c["pad"]:] = 0
        return dict(op="append", base=c["base"], interp=c["interp"], q=r.normal(T, Hq, D), k=r.normal(T, Hkv, D),
                    v=r.normal(T, Hkv, D), qg=r.gain(D), kg=r.gain(D), pos=i32(pos), slots=i32(slots),
                    k_pages=r.normal(n_pages, Hkv, P, D), v_pages=r.normal(n_pages, Hkv, P, D))
    L = _lengths(c, r)
    np_ = (L + c["P"] - 1) // c["P"]
    max_pages = int(np_.max())
    window = c.get("window", 0)
    first = ((L - window).clamp(min=0) // c["P"]) if window else torch.zeros_like(L)
    table, n_pages = _table(r, np_ - first, first, max_pages)
    s = dict(op=c["op"], P=c["P"], table=table, lens=i32(L))
    if c["op"] == "bounds":
        n_pages = c["B"] * (-(-c["hi"] // c["P"]))  # a pool of one size for every seed
        # Keys that share a direction within a page, as neighbouring tokens do.
        k = r.normal(n_pages, c["Hkv"], c["P"], c["D"])
        k += r.normal(n_pages, c["Hkv"], 1, c["D"])
        s.update(k_pages=k, old=i32(L - 1 if c["step"] else torch.zeros_like(L)),
                 bounds=torch.zeros(n_pages, c["Hkv"], 2, c["D"], dtype=torch.int8, device="cuda"),
                 exps=torch.zeros(n_pages, c["Hkv"], dtype=torch.int8, device="cuda"))
        return s
    s["q_hat"] = r.normal(c["B"], c["Hq"], c["D"])
    if c["op"] == "select":
        # Bounds of pages whose keys are near a mean of their own: their largest and smallest of P normal values.
        mean, spread = r.normal(n_pages, c["Hkv"], c["D"]).float(), math.sqrt(2 * math.log(c["P"])) * 0.9
        mx = (mean + spread + 0.4 * r.normal(n_pages, c["Hkv"], c["D"]).float()) * 16
        mn = (mean - spread - 0.4 * r.normal(n_pages, c["Hkv"], c["D"]).float()) * 16
        s.update(n_select=c["n_select"], bounds=torch.stack([mx, mn], 2).round().clamp(-127, 127).to(torch.int8),
                 exps=(4 - torch.randint(0, 2, (n_pages, c["Hkv"]), generator=r.g, device="cuda")).to(torch.int8))
        return s
    s.update(window=window, k_pages=r.normal(n_pages, c["Hkv"], c["P"], c["D"]),
             v_pages=r.normal(n_pages, c["Hkv"], c["P"], c["D"]), pages=None)
    if c["n_select"]:  # page lists as a selection gives them: ascending, the newest page last, -1 behind
        key = torch.rand(c["B"], c["Hkv"], max(max_pages, c["n_select"]), generator=r.g, device="cuda")
        at = torch.arange(key.shape[2], device="cuda")
        last = (np_ - 1).cuda()[:, None, None]
        key = torch.where(at == last, 2.0, torch.where(at < last, key, -1.0))
        val, idx = key.topk(c["n_select"], dim=2)
        idx = torch.where(val < 0, 1 << 30, idx).sort(dim=2).values
        s["pages"] = torch.where(idx == 1 << 30, -1, idx).to(torch.int32).contiguous()
    return s


# ------------------------------------------------------------- plain forms
def _plain_map(s):
    P, cap, T = s["P"], s["ring"].numel(), s["max_tokens"]
    old, new, max_pages = s["old"].long(), s["new"].long(), s["table"].shape[1]
    head, count = s["ring_state"].long()
    ends = new.cumsum(0)
    have = (old + P - 1) // P
    total = (old + new + P - 1) // P
    valid = (old + new <= max_pages * P) & (ends <= T)
    need = torch.where(valid, total - have, 0)
    cum = need.cumsum(0)
    granted = valid & ((need == 0) | (cum <= count))
    taken = torch.where(granted & (need > 0), cum, 0).max()
    lens = torch.where(granted, old + new, old)
    col = torch.arange(max_pages, device=old.device)
    fresh = granted[:, None] & (col >= have[:, None]) & (col < total[:, None])
    at = (head + (cum - need)[:, None] + col - have[:, None]) % cap
    table = torch.where(fresh, s["ring"][at], s["table"])
    t = torch.arange(T, device=old.device)
    b = torch.searchsorted(ends, t, right=True)
    inside = b < len(old)
    b = b.clamp(max=len(old) - 1)
    pos = old[b] + t - (ends[b] - new[b])
    ok = inside & granted[b]
    page = table[b, (pos // P).clamp(0, max_pages - 1)].long()
    slots = torch.where(ok & (page >= 0), page * P + pos % P, -1)
    cu = torch.cat([ends.new_zeros(1), ends]).clamp(max=T)
    s["table"].copy_(table)
    state = torch.stack([(head + taken) % cap, count - taken])
    i = torch.int32
    return dict(table=s["table"], seq_lens=lens.to(i), cu_tokens=cu.to(i), slots=slots.to(i),
                positions=torch.where(ok, pos, 0).to(i), free_state=state.to(i))


def _plain_norm_rope(x, gain, pos, base, interp):
    x = x.float()
    D = x.shape[-1]
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gain
    f = torch.arange(D // 2, dtype=torch.float64, device=x.device)
    theta = pos.double()[:, None] / interp * torch.pow(torch.tensor(base, dtype=torch.float64, device=x.device), -2 * f / D)
    cos, sin = theta.cos().float()[:, None], theta.sin().float()[:, None]
    a, b = y[..., :D // 2], y[..., D // 2:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(torch.bfloat16)


def _plain_append(s):
    q_hat = _plain_norm_rope(s["q"], s["qg"], s["pos"], s["base"], s["interp"])
    k_hat = _plain_norm_rope(s["k"], s["kg"], s["pos"], s["base"], s["interp"])
    P = s["k_pages"].shape[2]
    keep = s["slots"] >= 0
    slot = s["slots"].long()[keep]
    s["k_pages"][slot // P, :, slot % P] = k_hat[keep]
    s["v_pages"][slot // P, :, slot % P] = s["v"][keep]
    return dict(q_hat=q_hat, k_pages=s["k_pages"], v_pages=s["v_pages"])


def _exponent(amax):
    """The largest e with amax * 2^e <= 127, for a bf16 amax; within -50 .. 50."""
    m, x = torch.frexp(amax)  # amax = m * 2^x, 0.5 <= m < 1
    e = 7 - x - (m * 128 > 127).int()
    return torch.where(amax > 0, e, 50).clamp(-50, 50)


def _plain_bounds(s):
    P, table, L, old = s["P"], s["table"], s["lens"].long(), s["old"].long()
    col = torch.arange(table.shape[1], device=L.device)
    b, j = torch.nonzero((col >= (old // P)[:, None]) & (col < ((L + P - 1) // P)[:, None]), as_tuple=True)
    page = table[b, j].long()
    k = s["k_pages"][page].float()
    dead = (torch.arange(P, device=L.device) >= (L[b] - j * P)[:, None])[:, None, :, None]
    mx = k.masked_fill(dead, NEG).amax(2)
    mn = k.masked_fill(dead, -NEG).amin(2)
    e = _exponent(torch.maximum(mx.abs(), mn.abs()).amax(-1))
    scale = torch.ldexp(torch.ones_like(mx[..., :1]), e[..., None])
    s["bounds"][page] = torch.stack([(mx * scale).ceil(), (mn * scale).floor()], 2).clamp(-127, 127).to(torch.int8)
    s["exps"][page] = e.to(torch.int8)
    return dict(bounds=s["bounds"], exps=s["exps"])  # whole numbers by definition: equal, not near


def _plain_select(s):
    P, n, table, L = s["P"], s["n_select"], s["table"], s["lens"].long()
    B, Hq, D = s["q_hat"].shape
    Hkv = s["exps"].shape[1]
    q = s["q_hat"].float()
    e = _exponent(q.abs().amax(-1))
    q8 = torch.ldexp(q, e[..., None]).round().clamp(-127, 127).view(B, Hkv, -1, D)
    page = table.long().clamp(min=0)
    bnd = s["bounds"][page].float()                                     # [B, N, Hkv, 2, D]
    dot = torch.einsum("bhgd,bnhd->bhgn", q8.clamp(min=0), bnd[:, :, :, 0])
    dot = dot + torch.einsum("bhgd,bnhd->bhgn", q8.clamp(max=0), bnd[:, :, :, 1])
    score = torch.ldexp(dot, -e.view(B, Hkv, -1, 1) - s["exps"][page].int().permute(0, 2, 1)[:, :, None]).amax(2)
    last = ((L + P - 1) // P - 1)[:, None, None]
    at = torch.arange(table.shape[1], device=L.device)
    score = torch.where(at > last, NEG, torch.where(at == last, -NEG, score))
    val, idx = score.sort(dim=2, descending=True, stable=True)
    idx = torch.where(val == NEG, 1 << 30, idx)[:, :, :n].sort(dim=2).values
    out = torch.full((B, Hkv, n), -1, dtype=torch.int32, device=L.device)
    out[:, :, :idx.shape[2]] = torch.where(idx == 1 << 30, -1, idx)
    return out


def _plain_decode(s):
    P, table, L, W = s["P"], s["table"].long(), s["lens"].long(), s["window"]
    B, Hq, D = s["q_hat"].shape
    Hkv = s["k_pages"].shape[1]
    heads = torch.arange(Hkv, device=L.device)[None, :, None]
    if s["pages"] is not None:
        logical = s["pages"].long()                                     # [B, Hkv, N]
    else:
        n = table.shape[1]
        logical = torch.arange(n, device=L.device).expand(B, Hkv, -1)
        if W:                                                           # each row's own W tokens lie in its last pages
            n = min(n, (W + P - 2) // P + 1)
            logical = ((L + P - 1) // P - n).clamp(min=0)[:, None, None] + torch.arange(n, device=L.device).expand(B, Hkv, -1)
    tok = logical[..., None] * P + torch.arange(P, device=L.device)
    seen = (logical[..., None] >= 0) & (tok < L[:, None, None, None])
    if W:
        seen = seen & (tok >= (L - W)[:, None, None, None])
    phys = table[torch.arange(B, device=L.device)[:, None, None], logical.clamp(0, table.shape[1] - 1)].clamp(min=0)
    seen = seen.reshape(B, Hkv, 1, -1)
    q = s["q_hat"].float().view(B, Hkv, -1, D)
    K = s["k_pages"][phys, heads].view(B, Hkv, -1, D).float()
    x = (q @ K.transpose(2, 3) / math.sqrt(D)).masked_fill(~seen, NEG)
    del K
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp()
    total = p.sum(-1, keepdim=True)
    V = s["v_pages"][phys, heads].view(B, Hkv, -1, D).float()
    out = (p @ V / total).view(B, Hq, D).to(torch.bfloat16)
    return dict(out=out, lse=(m + total.log()).view(B, Hq))


_PLAIN = dict(map=_plain_map, append=_plain_append, bounds=_plain_bounds, select=_plain_select, decode=_plain_decode)


# -------------------------------------------------------- the framework's
def _own_map(s):
    got = _g3().page_map(s["old"], s["new"], s["table"], s["ring"], s["ring_state"], s["P"], s["n_pages"], s["max_tokens"])
    return dict(table=s["table"], seq_lens=got["seq_lens"], cu_tokens=got["cu_tokens"], slots=got["slots"],
                positions=got["positions"], free_state=got["free_state"])


def _own_append(s):
    q_hat = _g3().paged_append(s["k"], s["v"], s["kg"], s["pos"], s["slots"], s["k_pages"], s["v_pages"], s["base"],
                               s["interp"], q=s["q"], q_gamma=s["qg"])
    return dict(q_hat=q_hat, k_pages=s["k_pages"], v_pages=s["v_pages"])


def _own_bounds(s):
    _g3().page_bounds(s["k_pages"], s["table"], s["old"], s["lens"], s["bounds"], s["exps"])
    return dict(bounds=s["bounds"], exps=s["exps"])  # whole numbers by definition: equal, not near


def _own_select(s):
    return _g3().page_select(s["q_hat"], s["bounds"], s["exps"], s["table"], s["lens"], s["P"], s["n_select"])


def _own_decode(s):
    g3 = _g3()
    kind = g3.LOCAL if s["window"] else g3.GLOBAL
    out, lse = g3.paged_decode(s["q_hat"], s["k_pages"], s["v_pages"], s["table"], s["lens"], kind, s["window"],
                               pages=s["pages"], return_lse=True)
    return dict(out=out, lse=lse)


_OWN = dict(map=_own_map, append=_own_append, bounds=_own_bounds, select=_own_select, decode=_own_decode)


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# -------------------------------------------------------------------- work
def work(case):
    """Bytes and operations that a call cannot do without, at the case's mean lengths."""
    c = case
    if c["op"] == "map":
        mean_new = (c["new_lo"] + c["new_hi"]) / 2 * (c["B"] - c["idle"]) / c["B"]
        T = c["B"] * mean_new
        return dict(bytes=c["B"] * 16 + (c["B"] * c["new_hi"] + 13) * 8 + T / c["P"] * 8 + 16, flops=0)
    if c["op"] == "append":
        live, row = c["T"] - c["pad"], c["D"] * 2
        return dict(bytes=2 * (c["T"] * c["Hq"] + live * 2 * c["Hkv"]) * row + c["T"] * 8 + 8 * c["D"],
                    flops=(c["T"] * c["Hq"] + live * c["Hkv"]) * c["D"] * 7)
    L = ((c["lo"] + c["hi"]) / 2 * (c["B"] - 1) + c["hi"]) / c["B"]
    P, D, Hkv = c["P"], c["D"], c["Hkv"]
    pages = max(1.0, (L + (P - 1) / 2) / P)
    if c["op"] == "bounds":
        rows = (P + 1) / 2 if c["step"] else L
        n = 1 if c["step"] else pages
        return dict(bytes=c["B"] * Hkv * (rows * D * 2 + n * (2 * D + 1)) + c["B"] * 8 + c["B"] * n * 4, flops=0)
    if c["op"] == "select":
        return dict(bytes=c["B"] * (Hkv * pages * (2 * D + 1) + pages * 4 + c["Hq"] * D * 2 + Hkv * c["n_select"] * 4 + 4),
                    flops=2 * c["B"] * c["Hq"] * pages * D)
    seen = min(L, c["window"]) if c["window"] else min(L, c["n_select"] * P) if c["n_select"] else L
    return dict(bytes=c["B"] * (Hkv * seen * D * 4 + c["Hq"] * (D * 4 + 4) + seen / P * 4),
                flops=c["B"] * c["Hq"] * seen * D * 4)


# ---------------------------------------------------------- in 64 bits, apart
def _exact_map(s):
    import numpy as np
    n = lambda k: s[k].cpu().numpy().astype(np.int64)  # noqa: E731
    old, new, table, ring, (head, count) = n("old"), n("new"), n("table"), n("ring"), n("ring_state")
    P, T = s["P"], s["max_tokens"]
    slots, positions = np.full(T, -1, np.int32), np.zeros(T, np.int32)
    lens, cu, asked, taken, row = old.copy(), [0], 0, 0, 0
    for b in range(len(old)):
        have, total = -(-old[b] // P), -(-(old[b] + new[b]) // P)
        asked += total - have
        if total == have or asked <= count:
            for j in range(have, total):
                table[b, j] = ring[(head + asked - total + j) % len(ring)]
            if total > have:
                taken = asked
            lens[b] += new[b]
            p = np.arange(old[b], lens[b])
            slots[row:row + new[b]] = table[b, p // P] * P + p % P
            positions[row:row + new[b]] = p
        row += new[b]
        cu.append(row)
    i = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32))  # noqa: E731
    return dict(table=i(table), seq_lens=i(lens), cu_tokens=i(cu), slots=i(slots), positions=i(positions),
                free_state=i([(head + taken) % len(ring), count - taken]))


def _exact_append(s):
    def turned(x, gain):
        z = x.double()
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * gain.double()
        half = z.shape[-1] // 2
        z = torch.complex(z[..., :half], z[..., half:])
        w = torch.exp(torch.arange(half, device=z.device, dtype=torch.float64) * (-math.log(s["base"]) / half))
        ang = (s["pos"].double() / s["interp"])[:, None, None] * w
        z = z * torch.polar(torch.ones_like(ang), ang)
        return torch.cat([z.real, z.imag], -1)

    kh, kp, vp = turned(s["k"], s["kg"]), s["k_pages"].double(), s["v_pages"].double()
    n, Hkv, P, D = kp.shape
    live = torch.nonzero(s["slots"] >= 0).flatten()
    at = s["slots"][live].long()
    for pool, rows in ((kp, kh), (vp, s["v"].double())):
        flat = pool.transpose(1, 2).reshape(n * P, Hkv, D).clone()
        flat[at] = rows[live]
        pool.copy_(flat.view(n, P, Hkv, D).transpose(1, 2))
    return dict(q_hat=turned(s["q"], s["qg"]), k_pages=kp, v_pages=vp)


def _exact_bounds(s):
    P = s["P"]
    bounds, exps = s["bounds"].clone(), s["exps"].clone()
    for b in range(len(s["lens"])):
        L = int(s["lens"][b])
        j0, j1 = int(s["old"][b]) // P, -(-L // P)
        page = s["table"][b, j0:j1].long()
        k = s["k_pages"][page].double()
        hi, lo = k.clone(), k
        if L % P:
            hi[-1, :, L % P:], lo = -math.inf, k.clone()
            lo[-1, :, L % P:] = math.inf
        hi, lo = hi.max(2).values, lo.min(2).values
        e = torch.floor(torch.log2(127 / torch.maximum(hi.abs(), lo.abs()).max(-1).values)).clamp(-50, 50)
        unit = torch.exp2(e)[..., None]
        bounds[page] = torch.stack([torch.ceil(hi * unit), torch.floor(lo * unit)], 2).clamp(-127, 127).to(torch.int8)
        exps[page] = e.to(torch.int8)
    return dict(bounds=bounds, exps=exps)


def _exact_select(s):
    P, n = s["P"], s["n_select"]
    B, Hq, D = s["q_hat"].shape
    Hkv = s["exps"].shape[1]
    out = torch.full((B, Hkv, n), -1, dtype=torch.int32)
    q = s["q_hat"].double()
    eq = torch.floor(torch.log2(127 / q.abs().max(-1).values)).clamp(-50, 50)
    q = torch.round(q * torch.exp2(eq)[..., None]) * torch.exp2(-eq)[..., None]
    q = q.view(B, Hkv, Hq // Hkv, D)
    for b in range(B):
        N = -(-int(s["lens"][b]) // P)
        page = s["table"][b, :N].long()
        bnd = s["bounds"][page].double() * torch.exp2(-s["exps"][page].double())[..., None, None]   # [N, Hkv, 2, D]
        up = torch.where(q[b][None] >= 0, bnd[:, :, 0, None], bnd[:, :, 1, None])                    # [N, Hkv, G, D]
        score = (up * q[b][None]).sum(-1).max(-1).values.T                                           # [Hkv, N]
        score[:, N - 1] = math.inf
        order = torch.sort(-score, dim=1, stable=True).indices[:, :n]
        out[b, :, :order.shape[1]] = order.sort(1).values.cpu().to(torch.int32)
    return out


def _exact_decode(s):
    P = s["P"]
    B, Hq, D = s["q_hat"].shape
    Hkv = s["k_pages"].shape[1]
    out = torch.empty(B, Hq, D, dtype=torch.float64, device=s["q_hat"].device)
    lse = torch.empty(B, Hq, dtype=torch.float64, device=out.device)
    for b in range(B):
        L = int(s["lens"][b])
        lo = max(0, L - s["window"]) if s["window"] else 0
        for h in range(Hkv):
            if s["pages"] is None:
                tok = torch.arange(lo, L, device=out.device)
            else:
                j = s["pages"][b, h].long()
                tok = (j[j >= 0][:, None] * P + torch.arange(P, device=out.device)).flatten()
                tok = tok[tok < L]
            page = s["table"][b].long()[tok // P]
            g = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            z = s["k_pages"][page, h, tok % P].double() @ s["q_hat"][b, g].double().T / math.sqrt(D)
            lse[b, g] = torch.logsumexp(z, 0)
            out[b, g] = torch.exp(z - lse[b, g]).T @ s["v_pages"][page, h, tok % P].double()
    return dict(out=out, lse=lse)


def exact(case, seed):
    s = prepare(case, seed)
    return dict(map=_exact_map, append=_exact_append, bounds=_exact_bounds, select=_exact_select,
                decode=_exact_decode)[case["op"]](s)
