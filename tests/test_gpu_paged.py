"""Paged cache: page map, append, key bounds, page selection and single-token attention against the float64 oracle.

Tolerances are derived, not fitted.  A rounding to bf16 is off by at most 2^-8
of the value.  Whole-number results are equal.
  * q_hat and cached keys: one such rounding of y1 c - y2 s, whose fp32 terms
    are within 2^-18 of |y1| + |y2| (a sum of D squares, a reciprocal root, two
    products: some 30 roundings of 2^-24, 20 of them in the sum of squares).
  * decode: the output's rounding, 2^-8 |ref|, and P's, 2^-16 of each weight, which
    moves the output by at most 2^-16 times the weighted mean of |v|; the fp32 sums
    of q . k, at most (D + 8) 2^-24 of sum |q k| / sqrt D per exponent, move it by
    twice that share of the same mean, and those of P V, 2^-24 for each step of 16
    tokens and some 100 in the merges, by twice as much of it again.
  * lse: that bound on an exponent, and 2^-20 of its own size for the logarithm.
"""
import numpy as np
import pytest
import torch

import global_gqa_b200 as g3
import inputs
from oracle import attention as O
from oracle import paged as PG
from gpu_helpers import dev

pytestmark = pytest.mark.gpu

i32 = torch.int32


def gi(x):
    return torch.as_tensor(np.asarray(x), dtype=i32).to(dev())


def clean():
    """No device error has been recorded since the last check."""
    return g3.check_device_error(g3.paged_status(dev())) == 0


def reported():
    return g3.check_device_error(g3.paged_status(dev())) == 1


# --------------------------------------------------------------------- map
def run_map(old, new, table, ring, state, P, n_pages, T):
    """The call against the oracle, every output equal; returns the oracle's."""
    td, ref = gi(table), PG.page_map(old, new, table, ring, state, P, n_pages, T)
    got = g3.page_map(gi(old), gi(new), td, gi(ring), gi(state), P, n_pages, T)
    assert td.cpu().tolist() == ref["table"].tolist()
    for k in ("seq_lens", "cu_tokens", "slots", "positions", "free_state"):
        assert got[k].cpu().tolist() == ref[k].tolist(), k
    assert reported() if ref["error"] else clean()
    return ref


def random_map(rng, B, P, old_hi, new_hi, spare):
    old, new = rng.integers(0, old_hi + 1, B), rng.integers(0, new_hi + 1, B)
    new[rng.random(B) < 0.2] = 0
    have = -(-old // P)
    need = int((-(-(old + new) // P) - have).sum())
    max_pages = int((-(-(old + new) // P)).max()) + 1
    n_free = max(0, need + spare)
    n_pages = int(have.sum()) + n_free + 3
    perm = rng.permutation(n_pages)
    table, at = np.full((B, max_pages), -1), 0
    for b in range(B):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    ring = np.full(n_pages, -5)  # dead entries must not matter
    head = int(rng.integers(0, n_pages))
    ring[(head + np.arange(n_free)) % n_pages] = perm[at:at + n_free]
    return old, new, table, ring, [head, n_free], P, n_pages, int(new.sum()) + int(rng.integers(1, 40))


@pytest.mark.parametrize("B,P,old_hi,new_hi,spare", [
    (1, 16, 0, 1, 0), (1, 64, 1000, 70, 0), (3, 16, 40, 40, 5), (64, 64, 5000, 1, 9), (64, 128, 0, 700, 0),
    (1000, 16, 300, 33, 7), (1024, 32, 100, 1, 0), (1025, 32, 100, 3, 0), (2500, 256, 900, 5, 1), (8192, 16, 60, 2, 50),
    (7, 16, 100, 90, -6), (300, 32, 400, 60, -100), (40, 16, 50, 20, -1000),
])
def test_page_map(B, P, old_hi, new_hi, spare):
    for seed in range(3):
        run_map(*random_map(np.random.default_rng(seed * 1000 + B), B, P, old_hi, new_hi, spare))


@pytest.mark.parametrize("offset", [0, 1])
def test_page_map_long_buffer(offset):
    """More rows than threads: several per thread, also where the outputs are not aligned."""
    args = random_map(np.random.default_rng(offset), 600, 16, 100, 900, 3)
    old, new, table, ring, state, P, n_pages, T = args
    T = 200001
    td, ref = gi(table), PG.page_map(old, new, table, ring, state, P, n_pages, T)
    out = {k: torch.empty(T + 1, dtype=i32, device=dev())[offset:T + offset] for k in ("slots", "positions")}
    got = g3.page_map(gi(old), gi(new), td, gi(ring), gi(state), P, n_pages, T, out=out)
    assert (reported() if ref["error"] else clean()) and got["slots"] is out["slots"] and td.cpu().tolist() == ref["table"].tolist()
    for k in ("seq_lens", "cu_tokens", "slots", "positions", "free_state"):
        assert got[k].cpu().tolist() == ref[k].tolist(), k


def test_page_map_refuses_single_sequences():
    table, ring = np.full((6, 4), -1), np.arange(40)
    table[:, 0] = [30, 31, -1, 33, 99, 35]
    # negative lengths, a length past the table, a known page that is none, rows past the buffer
    run_map([5, -1, 0, 60, 3, 16], [3, 2, -4, 5, 2, 1], table, ring, [38, 40], 16, 50, 10)
    run_map([5, 3, 0, 16, 3, 16], [3, 2, 40, 5, 2, 1], table, ring, [0, 3], 16, 50, 48)
    run_map([2 ** 31 - 1, 0], [2 ** 31 - 1, 2 ** 31 - 1], np.full((2, 4), -1), ring, [0, 40], 16, 50, 10)


def test_page_map_bad_ring():
    args = [0, 16], [20, 1], np.array([[-1, -1, -1], [3, -1, -1]])
    run_map(*args, [9, 50, -2, 8], [0, 4], 16, 20, 30)   # page numbers that are none
    run_map(*args, [9, 5, 2, 8], [4, 4], 16, 20, 30)     # a head outside the ring
    run_map(*args, [9, 5, 2, 8], [0, 5], 16, 20, 30)     # a count above its size
    run_map(*args, [9, 5, 2, 8], [-1, 2], 16, 20, 30)


# ------------------------------------------------------------------ append
def append_inputs(T, Hq, Hkv, D, n_pages, P, seed, drop=0.1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    slots = torch.randperm(n_pages * P, generator=g)[:T]
    slots[torch.rand(T, generator=g) < drop] = -1
    return dict(q=r(T, Hq, D), k=r(T, Hkv, D), v=r(T, Hkv, D), qg=1 + 0.1 * torch.randn(D, generator=g),
                kg=1 + 0.1 * torch.randn(D, generator=g), pos=torch.randint(0, 131072, (T,), generator=g).to(i32),
                slots=slots.to(i32), kp=r(n_pages, Hkv, P, D), vp=r(n_pages, Hkv, P, D))


def near_rotated(got, x, gamma, pos, base, interp):
    ref, D = PG.norm_rope(x, gamma, pos, base, interp), x.shape[-1]
    y = np.abs(O.qk_rmsnorm(x, gamma))
    y = y[..., :D // 2] + y[..., D // 2:]
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * np.concatenate([y, y], -1)
    d = np.abs(got.double().cpu().numpy() - ref)
    assert (d <= tol).all(), float((d - tol).max())


@pytest.mark.parametrize("T,Hq,Hkv,D,P", [
    (1, 4, 2, 64, 16), (5, 32, 16, 128, 64), (64, 32, 16, 128, 64), (300, 4, 1, 256, 32), (64, 4, 1, 256, 128),
    (33, 24, 8, 128, 256), (700, 15, 3, 64, 16), (5000, 2, 2, 64, 128), (2400, 8, 1, 128, 16),
    (9, 40, 20, 128, 32), (21, 48, 9, 256, 16), (148, 64, 8, 128, 16), (149, 33, 16, 128, 64), (1184, 2, 1, 128, 16), (1185, 2, 1, 64, 16),
])
@pytest.mark.parametrize("with_q", [True, False])
def test_paged_append(T, Hq, Hkv, D, P, with_q):
    n_pages, base, interp = T // P + 3, (1e4 if D == 64 else 1e6), (1.0 if D == 64 else 8.0)
    x = append_inputs(T, Hq, Hkv, D, n_pages, P, T + D)
    d = {k: v.to(dev()) for k, v in x.items()}
    kw = dict(q=d["q"], q_gamma=d["qg"]) if with_q else {}
    q_hat = g3.paged_append(d["k"], d["v"], d["kg"], d["pos"], d["slots"], d["kp"], d["vp"], base, interp, **kw)
    assert clean()
    if with_q:
        near_rotated(q_hat, x["q"], x["qg"], x["pos"], base, interp)
    else:
        assert q_hat is None
    kp, vp = d["kp"].cpu(), d["vp"].cpu()
    live = x["slots"] >= 0
    s = x["slots"][live].long()
    near_rotated(kp[s // P, :, s % P], x["k"][live], x["kg"], x["pos"][live], base, interp)
    assert torch.equal(vp[s // P, :, s % P], x["v"][live])
    kp[s // P, :, s % P] = x["kp"][s // P, :, s % P]
    vp[s // P, :, s % P] = x["vp"][s // P, :, s % P]
    assert torch.equal(kp, x["kp"]) and torch.equal(vp, x["vp"])  # every other row as it was


def test_paged_append_zero_rows_and_bad_slots():
    x = append_inputs(6, 4, 2, 128, 2, 16, 3, drop=0)
    x["k"][1] = 0
    x["q"][2] = 0
    x["slots"] = torch.tensor([3, 31, 32, -1, 2 ** 31 - 1, -2 ** 31], dtype=i32)
    d = {k: v.to(dev()) for k, v in x.items()}
    q_hat = g3.paged_append(d["k"], d["v"], d["kg"], d["pos"], d["slots"], d["kp"], d["vp"], 1e6, 8.0, q=d["q"], q_gamma=d["qg"])
    assert reported() and clean()
    near_rotated(q_hat, x["q"], x["qg"], x["pos"], 1e6, 8.0)
    assert (d["kp"][1, :, 15] == 0).all() and torch.equal(d["vp"][0, :, 3].cpu(), x["v"][0])
    same = torch.ones(2, 16, dtype=torch.bool)
    same[0, 3] = same[1, 15] = False
    assert torch.equal(d["kp"].cpu().transpose(1, 2)[same], x["kp"].transpose(1, 2)[same])
    none = g3.paged_append(d["k"][:0], d["v"][:0], d["kg"], d["pos"][:0], d["slots"][:0], d["kp"], d["vp"], 1e6, 8.0,
                           q=d["q"][:0], q_gamma=d["qg"])
    assert none.shape == (0, 4, 128)


def test_append_writes_the_keys_that_prefill_caches():
    B, S, Hq, Hkv, D, P = 1, 200, 4, 2, 128, 32
    x = {k: v.to(dev()) for k, v in inputs.prefill_layer_inputs(B, S, Hq, Hkv, D, seed=3).items() if v is not None}
    kc, vc = (torch.zeros(B, Hkv, S, D, dtype=torch.bfloat16, device=dev()) for _ in "kv")
    g3.prefill(x["q"], x["k"], x["v"], x["q_gamma"], x["k_gamma"], x["positions"], g3.GLOBAL, 1024, 1e6, 8.0, k_cache=kc, v_cache=vc)
    kp, vp = (torch.zeros(7, Hkv, P, D, dtype=torch.bfloat16, device=dev()) for _ in "kv")
    g3.paged_append(x["k"][0], x["v"][0], x["k_gamma"], x["positions"][0], torch.arange(S, dtype=i32, device=dev()), kp, vp, 1e6, 8.0)
    flat = kp.transpose(0, 1).reshape(Hkv, -1, D)[:, :S]
    assert torch.equal(flat, kc[0]) and torch.equal(vp.transpose(0, 1).reshape(Hkv, -1, D)[:, :S], vc[0])


# ------------------------------------------------------------------ bounds
def scattered(rng, lens, P, extra=2, first=None):
    """A block table of randomly placed pages; entries before first[b] and behind the last are -1."""
    np_ = -(-np.asarray(lens) // P)
    first = np.zeros_like(np_) if first is None else first
    n_pages = int((np_ - first).sum()) + extra
    perm, table, at = rng.permutation(n_pages), np.full((len(lens), max(1, int(np_.max()))), -1), 0
    for b in range(len(lens)):
        n = np_[b] - first[b]
        table[b, first[b]:np_[b]] = perm[at:at + n]
        at += n
    return table, n_pages


def check_bounds(k_pages, table, old, lens, P):
    n_pages, Hkv, _, D = k_pages.shape
    bounds, exps = torch.full((n_pages, Hkv, 2, D), 99, dtype=torch.int8), torch.full((n_pages, Hkv), 99, dtype=torch.int8)
    ref, ref_e = bounds.clone(), exps.clone()
    for b, L in enumerate(lens):
        for j in range(old[b] // P, -(-L // P)):
            page = int(table[b, j])
            rows = min(P, L - j * P)
            for h in range(Hkv):
                bd, e = PG.page_bounds_of(k_pages[page, h, :rows])
                ref[page, h], ref_e[page, h] = torch.from_numpy(bd).to(torch.int8), e
    got, got_e = g3.page_bounds(k_pages.to(dev()), gi(table), gi(old), gi(lens), bounds.to(dev()), exps.to(dev()))
    assert torch.equal(got.cpu(), ref) and torch.equal(got_e.cpu(), ref_e)


@pytest.mark.parametrize("D,Hkv,P", [(64, 3, 16), (128, 2, 64), (256, 1, 32), (128, 16, 128), (64, 1, 256), (256, 4, 16)])
def test_page_bounds(D, Hkv, P):
    rng = np.random.default_rng(D + P)
    lens = [1, P - 1, P, P + 1, 3 * P + 5, 0, 2 * P]
    old = [0, P - 2, 0, P, P + 3, 0, 2 * P]
    table, n_pages = scattered(rng, lens, P)
    k = torch.randn(n_pages, Hkv, P, D, generator=torch.Generator().manual_seed(P)).bfloat16()
    k *= 2.0 ** torch.randint(-70, 70, (n_pages, Hkv, 1, 1), generator=torch.Generator().manual_seed(1))
    k[table[2, 0]] = 0
    k[table[4, 2], 0, 1] = k[table[4, 2], 0].max()  # a value that occurs twice
    for b, L in enumerate(lens):  # rows behind the last token must not matter
        if L % P:
            k[table[b, L // P], :, L % P:] = float("nan") if b % 2 else float("inf")
    check_bounds(k, table, old, lens, P)
    assert clean()


@pytest.mark.parametrize("D,P", [(64, 16), (64, 32), (128, 16)])
def test_page_bounds_many_small_pages(D, P):
    """More (page, kv head) pairs than one turn of the grid takes, some pages of them bad: 5 pairs a page, so that a
    warp's rows belong to different pages."""
    Hkv, n = 5, 4200
    rng = np.random.default_rng(D * P)
    k = torch.randn(n, Hkv, P, D, generator=torch.Generator().manual_seed(P)).bfloat16()
    lens, old = [n // 2 * P, n // 2 * P - P + 3], [0, P // 2]
    table = rng.permutation(n).reshape(2, n // 2)
    bad = [(0, 0), (0, 1), (0, 777), (1, 2), (1, n // 2 - 1)]
    for i, (b, j) in enumerate(bad):
        table[b, j] = [n, -1][i % 2]
    bounds, exps = torch.full((n, Hkv, 2, D), 99, dtype=torch.int8), torch.full((n, Hkv), 99, dtype=torch.int8)
    got, got_e = g3.page_bounds(k.to(dev()), gi(table), gi(old), gi(lens), bounds.to(dev()), exps.to(dev()))
    assert reported() and clean()
    rows = torch.full((2, n // 2), P)
    rows[1, -1] = 3
    for b in range(2):
        for j in range(n // 2):
            if (b, j) not in bad:
                for h in range(Hkv):
                    bd, e = PG.page_bounds_of(k[int(table[b, j]), h, :int(rows[b, j])])
                    bounds[int(table[b, j]), h], exps[int(table[b, j]), h] = torch.from_numpy(bd).to(torch.int8), e
    assert torch.equal(got.cpu(), bounds) and torch.equal(got_e.cpu(), exps)


def test_page_bounds_of_non_finite_and_extreme_keys():
    P, D = 16, 64
    k = torch.randn(4, 1, P, D, generator=torch.Generator().manual_seed(2)).bfloat16()
    k[0, 0, 3, 5] = float("nan")
    k[1, 0, 0, 0], k[1, 0, 1, 1] = float("inf"), -float("inf")
    k[2] *= 1e-30
    k[2, 0, :, 0] = 1e30
    k[3, 0, :, 1] = 127.5  # the largest mantissa
    k[3, 0, :, 2] = -1e-39
    check_bounds(k, np.arange(4)[:, None], [0] * 4, [16] * 4, P)
    assert clean()


def test_page_bounds_bad_pages_and_lengths():
    P, D = 16, 64
    k = torch.randn(3, 2, P, D, generator=torch.Generator().manual_seed(2)).bfloat16().to(dev())
    bounds, exps = torch.full((3, 2, 2, D), 99, dtype=torch.int8, device=dev()), torch.full((3, 2), 99, dtype=torch.int8, device=dev())
    for table, old, lens in (([[-1], [3]], [0, 0], [16, 5]), ([[0], [1]], [0, 0], [17, -1]), ([[0], [1]], [-1, 5], [3, 5 - 5])):
        g3.page_bounds(k, gi(table), gi(old), gi(lens), bounds, exps)
        assert reported() and (bounds == 99).all() and (exps == 99).all()


# ------------------------------------------------------------------ select
def check_select(q, bounds, exps, table, lens, P, n):
    B, Hkv = len(lens), exps.shape[1]
    got = g3.page_select(q.to(dev()), bounds.to(dev()), exps.to(dev()), gi(table), gi(lens), P, n).cpu().numpy()
    G = q.shape[1] // Hkv
    for b, L in enumerate(lens):
        page = table[b, :-(-L // P)]
        for h in range(Hkv):
            sc = PG.page_scores(q[b, h * G:(h + 1) * G], bounds[page, h].numpy(), exps[page, h].numpy())
            assert got[b, h].tolist() == PG.page_pick(sc, n).tolist(), (b, h)


@pytest.mark.parametrize("D,Hkv,G,P,n", [(64, 1, 1, 16, 1), (64, 2, 3, 16, 2), (128, 4, 2, 64, 5), (128, 2, 8, 32, 33),
                                         (256, 1, 4, 16, 64), (256, 3, 5, 128, 7), (128, 16, 2, 64, 1000)])
def test_page_select(D, Hkv, G, P, n):
    rng = np.random.default_rng(D + n)
    lens = [0, 1, P, n * P, n * P + 1, 70 * P, 65 * P + 3, 300 * P - 1]
    table, n_pages = scattered(rng, lens, P)
    g = torch.Generator().manual_seed(n)
    bounds = torch.randint(-127, 128, (n_pages, Hkv, 2, D), generator=g).sort(2, descending=True).values.to(torch.int8)
    exps = torch.randint(2, 5, (n_pages, Hkv), generator=g).to(torch.int8)
    check_select(torch.randn(len(lens), Hkv * G, D, generator=g).bfloat16(), bounds, exps, table, lens, P, n)
    assert clean()


def test_page_select_longest():
    """More pages than a block keeps the scores of: ties and a long list."""
    P, D, n = 16, 64, 1500
    rng, g = np.random.default_rng(8), torch.Generator().manual_seed(8)
    lens = [9000 * P, 6000 * P, 4096 * P, 4097 * P - 3, 8192 * P, 8193 * P - 3, 100]
    table, n_pages = scattered(rng, lens, P)
    bounds = torch.randint(-9, 10, (n_pages, 1, 2, D), generator=g).to(torch.int8)
    check_select(torch.randn(len(lens), 2, D, generator=g).bfloat16(), bounds, torch.full((n_pages, 1), 4, dtype=torch.int8), table, lens, P, n)
    check_select(torch.zeros(len(lens), 2, D).bfloat16(), bounds, torch.full((n_pages, 1), 4, dtype=torch.int8), table, lens, P, n)
    assert clean()


@pytest.mark.parametrize("D,Hkv,G,n", [(64, 4, 8, 7), (128, 8, 2, 64), (256, 3, 5, 1000), (128, 1, 1, 2)])
def test_page_select_few_long_sequences(D, Hkv, G, n):
    """Block tables of 1024 pages and more for few pairs; a short sequence beside the long one, equal scores in long runs."""
    P = 32
    rng, g = np.random.default_rng(D), torch.Generator().manual_seed(D)
    for lens in ([1024 * P], [2500 * P - 7, n * P], [1500 * P + 1, (n + 1) * P]):
        table, n_pages = scattered(rng, lens, P)
        q = torch.randn(len(lens), Hkv * G, D, generator=g).bfloat16()
        bounds = torch.randint(-127, 128, (n_pages, Hkv, 2, D), generator=g).to(torch.int8)
        exps = torch.randint(2, 6, (n_pages, Hkv), generator=g).to(torch.int8)
        check_select(q, bounds, exps, table, lens, P, n)
        bounds[torch.from_numpy(rng.permutation(n_pages)[:n_pages // 2])] = 5
        check_select(q, bounds, exps * 0 + 3, table, lens, P, n)
    assert clean()


@pytest.mark.parametrize("B", [100, 256, 300])
def test_page_select_many_sequences(B):
    """More pairs than find a place at once: taken by length, up to 256 sequences, equal and idle ones among them."""
    P, D, Hkv, n = 16, 128, 8, 4
    rng, g = np.random.default_rng(B), torch.Generator().manual_seed(B)
    lens = rng.integers(0, 30 * P, B)
    lens[::3] = 25 * P
    lens[1::5] = 0
    table, n_pages = scattered(rng, lens, P)
    bounds = torch.randint(-127, 128, (n_pages, Hkv, 2, D), generator=g).to(torch.int8)
    check_select(torch.randn(B, Hkv, D, generator=g).bfloat16(), bounds, torch.full((n_pages, Hkv), 4, dtype=torch.int8), table, lens, P, n)
    assert clean()
    lens[7], lens[11] = -5, 2 ** 31 - 1
    got = g3.page_select(torch.randn(B, Hkv, D, generator=g).bfloat16().to(dev()), bounds.to(dev()),
                         torch.full((n_pages, Hkv), 4, dtype=torch.int8, device=dev()), gi(table), gi(lens), P, n)
    assert reported() and (got[7] == -1).all() and (got[11] == -1).all() and (got[0, :, -1] == 24).all()


def test_page_select_ties_extremes_and_nan():
    P, D, Hkv, n = 16, 64, 2, 9
    rng, g = np.random.default_rng(5), torch.Generator().manual_seed(5)
    lens = [200 * P, 130 * P]
    table, n_pages = scattered(rng, lens, P)
    bounds = torch.randint(-3, 4, (4, 1, 2, D), generator=g).to(torch.int8)[torch.randint(0, 4, (n_pages,), generator=g)].repeat(1, Hkv, 1, 1)
    exps = torch.full((n_pages, Hkv), 3, dtype=torch.int8)
    q = torch.randn(2, 4, D, generator=g).bfloat16()
    check_select(q, bounds, exps, table, lens, P, n)                    # four kinds of pages: almost all scores are tied
    check_select(q * 0, bounds, exps, table, lens, P, n)                # every score is zero
    q[0, 0, 3], q[1, 2, 7], q[1, 3, 0] = float("nan"), float("inf"), -float("inf")
    exps[::3], exps[1::3] = -50, 50
    check_select(q, bounds, exps, table, lens, P, n)
    assert clean()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_page_select_largest_sums(D):
    """Sums of D products of 127 * 127 that differ by one unit in few places are told apart."""
    P, n = 16, 40
    rng = np.random.default_rng(D)
    table, n_pages = scattered(rng, [300 * P], P)
    for sign in (1, -1):
        q = sign * torch.full((1, 8, D), 127.0).bfloat16()
        q[0, 1:, ::2] *= -1
        bounds = torch.full((n_pages, 1, 2, D), 127, dtype=torch.int8)
        bounds[:, :, 1] = -127
        at = torch.from_numpy(rng.integers(0, D, n_pages))
        bounds[torch.arange(n_pages), 0, 0 if sign == 1 else 1, at] -= sign * torch.from_numpy(rng.integers(0, 3, n_pages)).to(torch.int8)
        check_select(q, bounds, torch.zeros(n_pages, 1, dtype=torch.int8), table, [300 * P], P, n)
        check_select(q, -bounds, torch.zeros(n_pages, 1, dtype=torch.int8), table, [300 * P], P, n)
    assert clean()


def test_page_select_bad_lengths_and_pages():
    P, D = 16, 64
    q = torch.randn(3, 2, D).bfloat16().to(dev())
    bounds, exps = torch.ones(6, 1, 2, D, dtype=torch.int8, device=dev()), torch.zeros(6, 1, dtype=torch.int8, device=dev())
    got = g3.page_select(q, bounds, exps, gi([[0, 1, 2]] * 3), gi([-1, 49, 40]), P, 2)
    assert reported() and (got[:2] == -1).all() and got[2, 0].tolist() == [0, 2]
    got = g3.page_select(q, bounds, exps, gi([[-1, 1, 2], [0, 6, 2], [0, 1, 2]]), gi([48] * 3), P, 2)
    assert reported() and got[:, 0].tolist() == [[1, 2], [0, 2], [0, 2]]  # a page that is none comes last


# ------------------------------------------------------------------ decode
def near_decode(out, lse, ref, D, longest):
    r, rl, mean_v, s_abs = ref
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    e = ((D + 8) * 2.0 ** -24 * s_abs)[..., None]
    tol = 2.0 ** -8 * np.abs(r) + (2.0 ** -16 + 2 * e + (longest / 8 + 200) * 2.0 ** -24) * (1 + 2.0 ** -7) * mean_v + 1e-30
    assert np.isfinite(got).all()
    assert (np.abs(got - r) <= tol).all(), float((np.abs(got - r) / tol).max())
    assert ((gl == -np.inf) == (rl == -np.inf)).all()
    seen = rl > -np.inf
    assert (np.abs(gl[seen] - rl[seen]) <= e[..., 0][seen] + 2.0 ** -20 * (1 + np.abs(rl[seen]))).all()
    assert (got[~seen] == 0).all()


def decode_case(lens, Hq, Hkv, D, P, seed, W=None, poison=True):
    """Pools in which everything that is not visible is NaN, and the call's arguments."""
    rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    lens = np.asarray(lens)
    first = None if W is None else np.maximum(0, lens - W) // P
    table, n_pages = scattered(rng, lens, P, first=first)
    kp, vp = (torch.randn(n_pages, Hkv, P, D, generator=g).bfloat16() for _ in "kv")
    if poison:
        live = torch.zeros(n_pages, P, dtype=torch.bool)
        for b, L in enumerate(lens):
            t = np.arange(max(0, L - W) if W else 0, L)
            live[table[b, t // P], t % P] = True
        kp.transpose(1, 2)[~live] = float("nan")
        vp.transpose(1, 2)[~live] = float("nan")
    return dict(q=torch.randn(len(lens), Hq, D, generator=g).bfloat16(), kp=kp, vp=vp, table=table, lens=lens)


def run_decode(c, kind=None, W=0, pages=None, **kw):
    kind = g3.GLOBAL if kind is None else kind
    out, lse = g3.paged_decode(c["q"].to(dev()), c["kp"].to(dev()), c["vp"].to(dev()), gi(c["table"]), gi(c["lens"]), kind, W,
                               pages=None if pages is None else gi(pages), return_lse=True, **kw)
    ref = PG.paged_decode(c["q"], c["kp"].double().numpy(), c["vp"].double().numpy(), c["table"], c["lens"], kind, W, pages)
    near_decode(out, lse, ref, c["q"].shape[2], int(np.max(c["lens"])))
    return out, lse


SHAPES = [(64, 1, 1, 16), (64, 2, 4, 64), (64, 3, 5, 16), (128, 2, 2, 64), (128, 4, 1, 16), (128, 1, 8, 32), (128, 8, 3, 128),
          (256, 1, 4, 64), (256, 2, 8, 16), (256, 1, 1, 256)]


@pytest.mark.parametrize("D,Hkv,G,P", SHAPES)
def test_paged_decode_all(D, Hkv, G, P):
    run_decode(decode_case([1, 2, 15, 16, 17, 0, P - 1, P, P + 1, 333, 1500], Hkv * G, Hkv, D, P, D + P))
    assert clean()
    run_decode(decode_case([4097], Hkv * G, Hkv, D, P, 1))      # one sequence over all blocks
    run_decode(decode_case([3], Hkv * G, Hkv, D, P, 2))
    run_decode(decode_case([0, 0], Hkv * G, Hkv, D, P, 3))
    run_decode(decode_case([9] * 257, Hkv * G, Hkv, D, P, 4))   # more pairs than blocks
    assert clean()


@pytest.mark.parametrize("D,Hkv,G,P", [(64, 8, 1, 16), (128, 16, 2, 32), (256, 8, 4, 16)])
def test_paged_decode_many_short(D, Hkv, G, P):
    """Pairs that are small parts of a block's share, beside idle sequences and one long one."""
    lens = np.random.default_rng(D).integers(0, 40, 1500)
    lens[::7], lens[700] = 0, 1200
    run_decode(decode_case(lens, Hkv * G, Hkv, D, P, 5))
    assert clean()


@pytest.mark.parametrize("B,hi", [(64, 18), (64, 70), (70, 130), (33, 33), (300, 50)])
@pytest.mark.parametrize("D,Hkv,G", [(64, 12, 2), (128, 16, 1), (256, 7, 8)])
def test_paged_decode_shares_of_few_pairs(B, hi, D, Hkv, G):
    """Blocks with a few pairs of one unit of 16 tokens, of two and of more, whole ones and cut ones, in any order."""
    run_decode(decode_case(np.random.default_rng(B + hi).integers(1, hi, B), Hkv * G, Hkv, D, 16, 6))
    assert clean()


@pytest.mark.parametrize("D,Hkv,G,P", SHAPES[::3])
@pytest.mark.parametrize("W", [1, 7, 16, 100, 1024, 5000])
def test_paged_decode_window(D, Hkv, G, P, W):
    run_decode(decode_case([1, 16, 100, 101, 1024, 1025, 2049, 0, 3001], Hkv * G, Hkv, D, P, W, W=W), kind=g3.LOCAL, W=W)
    assert clean()  # table entries before the window are -1 and are not read


@pytest.mark.parametrize("D,Hkv,G,P", SHAPES[1::3])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_paged_decode_selected(D, Hkv, G, P, n):
    rng = np.random.default_rng(n)
    lens = np.array([1, P, P + 1, 5 * P, 5 * P - 3, 0, 60 * P + 9])
    c = decode_case(lens, Hkv * G, Hkv, D, P, n)
    pages = np.full((len(lens), Hkv, n), -1)
    for b, L in enumerate(lens):
        for h in range(Hkv):
            N = -(-L // P)
            if N:
                pick = sorted(rng.permutation(N - 1)[:n - 1].tolist()) + [N - 1]
                pages[b, h, :len(pick)] = pick
    run_decode(c, pages=pages)
    assert clean()
    pages[:, :, 0] = np.where(pages[:, :, 1:2].max(2) >= 0, pages[:, :, 0], -1) if n > 1 else -1
    run_decode(c, pages=pages)  # lists with nothing in them
    assert clean()


def test_paged_decode_full_size_sampled():
    """64 sequences of 4K to 32K tokens, 27B heads: six sequences against the oracle, the rest by equal sequences."""
    Hq, Hkv, D, P = 32, 16, 128, 64
    rng = np.random.default_rng(0)
    lens = rng.integers(4096, 32769, 64)
    table, n_pages = scattered(rng, lens, P)
    kp = torch.empty(n_pages, Hkv, P, D, dtype=torch.bfloat16, device=dev())
    vp = torch.empty_like(kp)
    inputs.device_fill_normal_bf16(kp, 1)
    inputs.device_fill_normal_bf16(vp, 2)
    q = torch.randn(64, Hq, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    out, lse = g3.paged_decode(q.to(dev()), kp, vp, gi(table), gi(lens), g3.GLOBAL, 0, return_lse=True)
    for b in (0, 1, 31, 62, 63, int(np.argmax(lens))):
        n = -(-int(lens[b]) // P)
        idx = torch.as_tensor(table[b, :n], device=dev(), dtype=torch.long)
        ref = PG.paged_decode(q[b:b + 1], kp[idx].double().cpu().numpy(), vp[idx].double().cpu().numpy(), np.arange(n)[None],
                              lens[b:b + 1], 1, 0)
        near_decode(out[b:b + 1], lse[b:b + 1], ref, D, int(lens[b]))
        one = g3.paged_decode(q[b:b + 1].to(dev()), kp, vp, gi(table[b:b + 1]), gi(lens[b:b + 1]), g3.GLOBAL, 0)
        near_decode(one, lse[b:b + 1], ref, D, int(lens[b]))  # cut in other places
    assert clean()


def test_paged_decode_repeats_bit_for_bit():
    c = decode_case([5000, 77, 4096, 1], 8, 2, 128, 32, 9)
    a = run_decode(c)
    for _ in range(3):
        b = run_decode(c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_paged_decode_extreme_scores():
    c = decode_case([40, 700], 4, 2, 64, 16, 1)
    c["q"] *= 100   # weights of nearly one and nearly zero
    run_decode(c)
    c["vp"][c["table"][0, 0], 0, 5, 7] = float("inf")
    out, _ = g3.paged_decode(c["q"].to(dev()), c["kp"].to(dev()), c["vp"].to(dev()), gi(c["table"]), gi(c["lens"]), g3.GLOBAL, 0,
                             return_lse=True)
    assert not torch.isfinite(out[0, :2, 7]).any() and torch.isfinite(out[0, :2, 8:]).all() and torch.isfinite(out[0, 2:]).all()
    c["kp"][c["table"][1, 3], 1, 2, 9] = float("nan")  # a NaN that is seen makes its heads NaN
    out, lse = g3.paged_decode(c["q"].to(dev()), c["kp"].to(dev()), c["vp"].to(dev()), gi(c["table"]), gi(c["lens"]), g3.GLOBAL, 0,
                               return_lse=True)
    assert torch.isnan(out[1, 2:]).all() and torch.isnan(lse[1, 2:]).all() and torch.isfinite(out[1, :2]).all()


def test_paged_decode_bad_pages_lengths_and_lists():
    c = decode_case([100, 64, 30], 4, 2, 64, 16, 5)
    lens = c["lens"].copy()
    c["table"][0, 2], c["table"][1, 0] = -1, c["kp"].shape[0]
    run_decode(c)                                   # the oracle leaves the same pages out
    assert reported()
    c["table"] = decode_case([100, 64, 30], 4, 2, 64, 16, 5)["table"]
    c["lens"] = np.array([-3, c["table"].shape[1] * 16 + 1, 30])
    run_decode(c)
    assert reported() and clean()
    c["lens"] = lens
    bad = np.array([[[0, 0, 3], [1, 9, 2]], [[3, 2, -1], [-7, 1, 2]], [[0, 1, 2], [0, 1, -1]]])
    good = np.array([[[0, -1, 3], [1, -1, 2]], [[3, -1, -1], [-1, 1, 2]], [[0, 1, -1], [0, 1, -1]]])
    got = g3.paged_decode(c["q"].to(dev()), c["kp"].to(dev()), c["vp"].to(dev()), gi(c["table"]), gi(lens), g3.GLOBAL, 0, pages=gi(bad))
    assert reported()
    # [1, 9, 2]: 9 is past the sequence and 2 is not above it; the oracle's list without what is left out
    good[0, 1] = [1, -1, -1]
    ref = PG.paged_decode(c["q"], c["kp"].double().numpy(), c["vp"].double().numpy(), c["table"], lens, 1, 0, good)
    near_decode(got, torch.from_numpy(ref[1]), ref, 64, 100)


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements: append, bounds, selection and decode in its last pages."""
    Hkv, G, D, P = 16, 2, 128, 64
    n_pages = (1 << 31) // (Hkv * P * D) + 40
    kp = torch.zeros(n_pages, Hkv, P, D, dtype=torch.bfloat16, device=dev())
    vp = torch.zeros_like(kp)
    L, last = 200, n_pages - 1
    table = np.array([[last, 3, last - 7, last - 1]])
    x = append_inputs(L, Hkv * G, Hkv, D, 1, 256, 1, drop=0)
    t = np.arange(L)
    slots = table[0, t // P] * P + t % P
    d = {k: x[k].to(dev()) for k in ("q", "k", "v", "qg", "kg")}
    q_hat = g3.paged_append(d["k"], d["v"], d["kg"], gi(t), gi(slots), kp, vp, 1e6, 8.0, q=d["q"], q_gamma=d["qg"])
    idx = torch.as_tensor(table[0], device=dev(), dtype=torch.long)
    k_small, v_small = kp[idx].cpu(), vp[idx].cpu()
    near_rotated(k_small.transpose(1, 2).reshape(-1, Hkv, D)[:L], x["k"], x["kg"], t, 1e6, 8.0)
    bounds, exps = torch.zeros(n_pages, Hkv, 2, D, dtype=torch.int8, device=dev()), torch.zeros(n_pages, Hkv, dtype=torch.int8, device=dev())
    g3.page_bounds(kp, gi(table), gi([0]), gi([L]), bounds, exps)
    bd, e = PG.page_bounds_of(k_small[3, 15, :L - 3 * P])
    assert bounds[last - 1, 15].cpu().tolist() == bd.tolist() and int(exps[last - 1, 15]) == e
    pages = g3.page_select(q_hat[-1:], bounds, exps, gi(table), gi([L]), P, 3)
    out, lse = g3.paged_decode(q_hat[-1:], kp, vp, gi(table), gi([L]), g3.GLOBAL, 0, pages=pages, return_lse=True)
    ref = PG.paged_decode(q_hat[-1:].cpu(), k_small.double().numpy(), v_small.double().numpy(), np.arange(4)[None], [L], 1, 0,
                          pages.cpu().numpy())
    near_decode(out, lse, ref, D, L)
    assert clean()
