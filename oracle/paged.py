"""Plain float64 definitions of the paged-cache operators (test infrastructure).

Loops over sequences, heads and pages as include/g3attn.h words them; shares no
code with the CUDA library.  The norm, the rotation and the softmax are those of
oracle/attention.py.
"""
from __future__ import annotations

import math

import numpy as np

from .attention import _f64, _i64, qk_rmsnorm, rope


def page_map(old_lens, new_lens, block_table, free_pages, free_state, page_size, n_pages, max_tokens):
    """dict(table, seq_lens, cu_tokens, slots, positions, free_state, error): one request after the other."""
    P, cap = page_size, len(free_pages)
    table = np.array(block_table, dtype=np.int64)
    head, count = (int(x) for x in free_state)
    error = False
    if not (0 <= head < cap and 0 <= count <= cap):
        head, count, error = 0, 0, True
    slots, positions = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int64)
    lens, cu, row, asked, taken = [], [0], 0, 0, 0
    room = table.shape[1] * P
    for b, (old, new) in enumerate(zip(_i64(old_lens).tolist(), _i64(new_lens).tolist())):
        row0, row = row, row + max(new, 0)
        cu.append(min(row, max_tokens))
        valid = old >= 0 and new >= 0 and old + new <= room and row <= max_tokens
        granted = False
        if valid:
            have, total = -(-old // P), -(-(old + new) // P)
            asked += total - have
            granted = total == have or asked <= count
        error |= not granted
        lens.append(old + new if granted else old if 0 <= old <= room else 0)
        if not granted:
            continue
        for j in range(have, total):
            page = int(free_pages[(head + asked - total + j) % cap])
            if not 0 <= page < n_pages:
                page, error = -1, True
            table[b, j] = page
        if total > have:
            taken = asked
        for i in range(new):
            page = int(table[b, (old + i) // P])
            positions[row0 + i] = old + i
            if 0 <= page < n_pages:
                slots[row0 + i] = page * P + (old + i) % P
            else:
                error = True
    return dict(table=table, seq_lens=np.array(lens), cu_tokens=np.array(cu), slots=slots, positions=positions,
                free_state=np.array([(head + taken) % cap, count - taken]), error=error)


def norm_rope(x, gamma, positions, base, interp):
    """Normalised and rotated rows of x [T, H, D] (float64)."""
    return rope(qk_rmsnorm(_f64(x), gamma), _f64(positions), base, interp)


def exponent(amax: float) -> int:
    """The largest e within -50 .. 50 with amax * 2^e <= 127."""
    if amax == 0:
        return 50
    if not math.isfinite(amax):
        return -50
    e = 50
    while e > -50 and math.ldexp(amax, e) > 127:
        e -= 1
    return e


def page_bounds_of(rows):
    """(bounds [2, D], e) of one page's filled key rows [n, D]."""
    rows = _f64(rows)
    bad = np.isnan(rows).any(0)
    big, small = rows.max(0), rows.min(0)
    e = exponent(math.inf if bad.any() else float(np.maximum(np.abs(big), np.abs(small)).max()))
    with np.errstate(invalid="ignore"):
        up = np.clip(np.ceil(np.ldexp(big, e)), -127, 127)
        down = np.clip(np.floor(np.ldexp(small, e)), -127, 127)
    up[bad], down[bad] = 127, -127
    return np.stack([up, down]).astype(np.int64), e


def page_scores(q, bounds, exps):
    """Scores [N] of one (sequence, kv head): q [G, D], bounds [N, 2, D] whole numbers, exps [N]."""
    q = np.nan_to_num(_f64(q), nan=0.0, posinf=math.inf, neginf=-math.inf)
    best = np.full(len(exps), -math.inf)
    for row in q:
        e = exponent(float(np.abs(row).max()))
        q8 = np.clip(np.rint(np.ldexp(row, e)), -127, 127)
        dot = np.maximum(q8, 0) @ _f64(bounds)[:, 0].T + np.minimum(q8, 0) @ _f64(bounds)[:, 1].T
        best = np.maximum(best, np.ldexp(dot, -e - _i64(exps)))
    return best


def page_pick(scores, n_select):
    """Logical pages of one (sequence, kv head): the last and the n_select - 1 best others, ascending, -1 behind."""
    n = len(scores)
    if n == 0:
        return np.full(n_select, -1)
    others = sorted(range(n - 1), key=lambda j: (-scores[j], j))[:n_select - 1]
    got = sorted(others) + [n - 1]
    return np.array(got + [-1] * (n_select - len(got)))


def paged_decode(q_hat, k_pages, v_pages, block_table, seq_lens, kind, window, pages=None):
    """out [B, Hq, D], lse [B, Hq], and per (b, head) two magnitudes that bound a kernel's rounding:
    mean |v| under the softmax weights [B, Hq, D] and the largest sum |q||k| / sqrt(D) [B, Hq]."""
    q = _f64(q_hat)
    B, Hq, D = q.shape
    n_pages, Hkv, P, _ = k_pages.shape
    G = Hq // Hkv
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    mean_v, s_abs = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    table = _i64(block_table)
    for b, L in enumerate(_i64(seq_lens).tolist()):
        if not 0 < L <= table.shape[1] * P:
            continue
        for h in range(Hkv):
            lo = max(0, L - window) if kind == 0 and pages is None else 0
            logical = np.arange(lo // P, -(-L // P)) if pages is None else _i64(pages)[b, h]
            toks = (logical[logical >= 0][:, None] * P + np.arange(P)).ravel()
            toks = toks[(toks >= lo) & (toks < L)]
            phys = table[b, toks // P]
            toks, phys = toks[(phys >= 0) & (phys < n_pages)], phys[(phys >= 0) & (phys < n_pages)]
            if toks.size == 0:
                continue
            K, V = _f64(k_pages[phys, h, toks % P]), _f64(v_pages[phys, h, toks % P])
            for g in range(h * G, (h + 1) * G):
                s = K @ q[b, g] / math.sqrt(D)
                m = s.max()
                p = np.exp(s - m)
                out[b, g] = p @ V / p.sum()
                lse[b, g] = m + math.log(p.sum())
                mean_v[b, g] = p @ np.abs(V) / p.sum()
                s_abs[b, g] = (np.abs(K) @ np.abs(q[b, g])).max() / math.sqrt(D)
    return out, lse, mean_v, s_abs
