"""What the paged calls' documentation promises at the edges of their arguments, one promise per test.

Tolerances are those that test_gpu_paged.py derives."""
import numpy as np
import pytest
import torch

import global_gqa_b200 as g3
import inputs
from oracle import paged as PG
from gpu_helpers import dev
from test_gpu_paged import check_select, clean, decode_case, gi, near_decode, reported, scattered
from test_gpu_paged_serving import Pool, Step, layer, near, same

pytestmark = pytest.mark.gpu
i32 = torch.int32


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("D,Hkv,G,P", [(64, 2, 2, 16), (128, 2, 3, 32), (256, 1, 4, 16)])
@pytest.mark.parametrize("lens", [[1, 40, 700], [4097], [9, 33, 1200] + [5, 20] * 400], ids=["few", "one", "many"])
def test_infinite_values_stay_infinite(D, Hkv, G, P, lens):
    """An infinity in a visible V row makes its feature that infinity whatever the row's weight, both signs a NaN, and no other feature
    differs from what it is without them: pairs cut between blocks, whole ones, single warps' ones."""
    c = decode_case(lens, Hkv * G, Hkv, D, P, 11)
    call = lambda: g3.paged_decode(c["q"].to(dev()), c["kp"].to(dev()), c["vp"].to(dev()), gi(c["table"]), gi(c["lens"]), g3.GLOBAL, 0,  # noqa: E731
                                   return_lse=True)
    plain, plain_lse = call()
    for b, L in enumerate(lens):
        for f, t, v in ((3, 0, np.inf), (D // 2, L - 1, -np.inf), (D - 1, L // 2, np.inf)):
            c["vp"][c["table"][b, t // P], Hkv - 1, t % P, f] = v
        if L > 1:  # both signs
            for t, v in ((0, np.inf), (L - 1, -np.inf)):
                c["vp"][c["table"][b, t // P], Hkv - 1, t % P, 7] = v
    out, lse = call()
    hit = out[:, (Hkv - 1) * G:]
    assert (hit[..., 3] == np.inf).all() and (hit[..., D // 2] == -np.inf).all() and (hit[..., D - 1] == np.inf).all()
    assert torch.isnan(hit[np.asarray(lens) > 1][..., 7]).all()
    left = torch.ones_like(out, dtype=torch.bool)
    left[:, (Hkv - 1) * G:, [3, 7, D // 2, D - 1]] = False
    assert torch.equal(out[left], plain[left]) and torch.equal(lse, plain_lse) and clean()


def test_infinite_values_of_small_weights():
    """Weights down to 2^-86 of the largest, and one of exactly a power of two."""
    P, D, L = 16, 64, 40
    c = decode_case([L], 1, 1, D, P, 3)
    c["q"][:] = 0
    c["q"][0, 0, 0] = 64
    c["kp"][..., 0] = 0
    for t, k in ((0, -7.5), (20, 0.0), (33, -4.0)):  # exponents 8 k: weights e^-60, 1, e^-32
        c["kp"][c["table"][0, t // P], 0, t % P, 0] = k
        c["vp"][c["table"][0, t // P], 0, t % P, t] = np.inf
    out = g3.paged_decode(c["q"].to(dev()), c["kp"].to(dev()), c["vp"].to(dev()), gi(c["table"]), gi(c["lens"]), g3.GLOBAL, 0)
    assert (out[0, 0, [0, 20, 33]] == np.inf).all() and int(torch.isfinite(out).sum()) == D - 3 and clean()


def test_list_entries_behind_a_pad():
    """An entry is compared with the one before it alone: pages behind a -1 are attended to, one listed again counts again; entries behind
    the sequence's number of pages are not read."""
    L, P, D = 96, 16, 64
    c = decode_case([L, L, 2 * P], 2, 1, D, P, 5)
    listed = np.array([[[5, -1, 5, -1]], [[0, -1, 4, -1]], [[0, 1, 0, 9]]])
    ref = PG.paged_decode(c["q"], c["kp"].double().numpy(), c["vp"].double().numpy(), c["table"], c["lens"], 1, 0, listed[:, :, :3] * 1)
    one = PG.paged_decode(c["q"][2:], c["kp"].double().numpy(), c["vp"].double().numpy(), c["table"][2:], c["lens"][2:], 1, 0)
    for r, o in zip(ref, one):
        r[2] = o[0]
    out, lse = g3.paged_decode(c["q"].to(dev()), c["kp"].to(dev()), c["vp"].to(dev()), gi(c["table"]), gi(c["lens"]), g3.GLOBAL, 0,
                               pages=gi(listed), return_lse=True)
    near_decode(out, lse, ref, D, L)
    assert clean()


@pytest.mark.parametrize("flag", [1, np.bool_(True), 0, np.bool_(False), None, True, False])
def test_lse_is_returned_alike_by_both_ways_of_the_call(flag):
    c = decode_case([5, 20], 2, 1, 64, 16, 1)
    args = c["q"].to(dev()), c["kp"].to(dev()), c["vp"].to(dev()), gi(c["table"]), gi(c["lens"]), g3.GLOBAL, 0
    quick = g3.paged_decode(*args, return_lse=flag)
    ordinary = g3.paged_decode(*args, return_lse=flag, out=torch.empty_like(args[0]))
    assert isinstance(quick, tuple) == isinstance(ordinary, tuple) == bool(flag)
    for a, b in zip(quick, ordinary):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ bounds
def test_no_new_tokens_renew_no_bounds():
    """old == seq_len, or above it, inside a page and at its border: nothing is read, written or recorded."""
    P, D = 16, 64
    k = torch.randn(8, 2, P, D, generator=torch.Generator().manual_seed(2)).bfloat16().to(dev())
    bounds, exps = torch.full((8, 2, 2, D), 99, dtype=torch.int8, device=dev()), torch.full((8, 2), 99, dtype=torch.int8, device=dev())
    old, lens = [5, 20, 30, 16, 20, 31, 0, 32], [5, 20, 20, 16, 3, 17, 0, 32]
    for page in (-1, 0, 8):  # also where the table holds no page
        g3.page_bounds(k, gi(np.full((8, 2), page)), gi(old), gi(lens), bounds, exps)
        assert clean() and (bounds == 99).all() and (exps == 99).all()
    table = np.arange(8).reshape(4, 2)
    g3.page_bounds(k, gi(table), gi([5, 20, 7, 32]), gi([5, 21, 7, 32]), bounds, exps)  # one of four has a token
    assert clean() and (bounds[[0, 1, 2, 4, 5, 6, 7]] == 99).all()
    for h in range(2):
        ref, e = PG.page_bounds_of(k[3, h, :5].cpu())
        assert bounds[3, h].cpu().tolist() == ref.tolist() and int(exps[3, h]) == e


# ------------------------------------------------------------------ select
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B", [2, 24])
def test_page_select_of_more_pages_than_fit_on_chip(D, B):
    """Block tables above 8192 pages, scores in the workspace: few pairs (blocks of 512 threads) and more (of 256)."""
    P, n, n_pages = 16, 100, 700
    rng, g = np.random.default_rng(B + D), torch.Generator().manual_seed(B + D)
    lens = rng.integers(100 * P, 8193 * P, B)
    lens[0], lens[-1] = 8500 * P - 3, 8193 * P
    table = rng.integers(0, n_pages, (B, 8500))
    bounds = torch.randint(-127, 128, (n_pages, 1, 2, D), generator=g).to(torch.int8)
    exps = torch.randint(2, 5, (n_pages, 1), generator=g).to(torch.int8)
    check_select(torch.randn(B, 3, D, generator=g).bfloat16(), bounds, exps, table, lens, P, n)  # pages repeat: many ties
    assert clean()


@pytest.mark.parametrize("D,B", [(256, 150), (256, 295), (128, 296), (256, 148), (64, 148), (256, 74)])
def test_page_select_pairs_around_the_clusters_limits(D, B):
    P, n, n_pages = 16, 9, 700
    rng, g = np.random.default_rng(B + D), torch.Generator().manual_seed(B + D)
    lens = rng.integers(0, 600 * P, B)
    table = rng.integers(0, n_pages, (B, 600))
    bounds = torch.randint(-127, 128, (n_pages, 1, 2, D), generator=g).to(torch.int8)
    check_select(torch.randn(B, 2, D, generator=g).bfloat16(), bounds, torch.full((n_pages, 1), 4, dtype=torch.int8), table, lens, P, n)
    assert clean()


# --------------------------------------------------------------------- map
@pytest.mark.parametrize("T", [4, 8192, 8193, 100000])
def test_kept_lengths_hold_few_token_rows(T):
    """What a server keeps from step to step does not keep a prompt's slots and positions alive: 64 KB of them at most."""
    B = 4
    got = g3.page_map(gi([0] * B), gi([1] * B), gi(np.full((B, 2), -1)), gi(np.arange(9)), gi([0, 9]), 16, 9, T)
    for k in ("seq_lens", "cu_tokens", "free_state"):
        assert got[k].untyped_storage().nbytes() <= 2 * 4 * 8192 + 4096
    places = sorted((got[k].data_ptr(), got[k].data_ptr() + got[k].numel() * 4) for k in got)
    assert all(a[1] <= b[0] and b[0] % 256 == 0 for a, b in zip(places, places[1:]))
    assert got["seq_lens"].tolist() == [1] * B and got["cu_tokens"].tolist() == [0, 1, 2, 3, 4] and got["free_state"].tolist() == [4, 5]
    assert got["slots"][:4].tolist() == [0, 16, 32, 48] and (got["slots"][4:] == -1).all() and (got["positions"] == 0).all() and clean()


# ----------------------------------------------------------------- serving
def newest_rows(q_hat, cu_tokens):
    """The packed rows of each sequence's newest token, as the documentation gathers them."""
    return q_hat.index_select(0, (cu_tokens[1:] - 1).clamp(min=0))


@pytest.mark.parametrize("Hq,Hkv,D,P", [(4, 2, 64, 16), (8, 2, 128, 32), (4, 1, 256, 16)])
def test_sequences_with_a_history_wait_a_step(Hq, Hkv, D, P):
    """Steps in which some sequences get no token: the others' results are those of the contiguous decode, and what
    belongs to a waiting one (table, length, pages, bounds) is left as it was."""
    B, W, cap, n_pages = 4, 48, 200, 60
    pool = Pool(2, n_pages, B, -(-cap // P), Hkv, D, P)
    ring = [[torch.zeros(B, Hkv, W if li == 0 else cap, D, dtype=torch.bfloat16, device=dev()) for _ in "kv"] for li in range(2)]
    gains = [inputs.prefill_layer_inputs(1, 1, Hq, Hkv, D, seed=0, layer=li) for li in range(2)]
    gains = [(x["q_gamma"].to(dev()), x["k_gamma"].to(dev())) for x in gains]
    prompts = [70, 31, 50, 33]
    got = pool.map(prompts, sum(prompts))
    for li in range(2):
        kind, win, base, interp = layer(li, W)
        packed = [torch.empty(sum(prompts), Hkv, D, dtype=torch.bfloat16, device=dev()) for _ in "kv"]
        for b, n in enumerate(prompts):
            x = {k: v.to(dev()) for k, v in inputs.prefill_layer_inputs(1, n, Hq, Hkv, D, seed=60 + b, layer=li).items() if v is not None}
            kc, vc = ring[li][0][b:b + 1], ring[li][1][b:b + 1]
            g3.prefill(x["q"], x["k"], x["v"], *gains[li], x["positions"], kind, win, base, interp, k_cache=kc, v_cache=vc)
            r0 = int(got["cu_tokens"][b])
            packed[0][r0:r0 + n], packed[1][r0:r0 + n] = x["k"][0], x["v"][0]
        g3.paged_append(*packed, gains[li][1], got["positions"], got["slots"], pool.k[li], pool.v[li], base, interp)
    g3.page_bounds(pool.k[1], pool.table, pool.old, pool.lens, pool.bounds, pool.exps)

    for s, active in enumerate([[1, 0, 1, 1], [0, 1, 1, 1], [1, 1, 1, 0], [0, 0, 1, 0], [1, 0, 0, 1], [0, 0, 0, 0], [1, 1, 1, 1]] * 3):
        rows, waiting = [b for b in range(B) if active[b]], [b for b in range(B) if not active[b]]
        before = pool.table.clone(), pool.lens.clone(), pool.bounds.clone(), pool.exps.clone(), [k.clone() for k in pool.k + pool.v]
        theirs = torch.cat([pool.table[b, :-(-int(pool.lens[b]) // P)] for b in waiting]).long() if waiting else torch.empty(0, dtype=torch.long)
        got = pool.map(active, B)
        for li in range(2):
            kind, win, base, interp = layer(li, W)
            x = {k: v.to(dev()) for k, v in inputs.decode_step_inputs(B, Hq, Hkv, D, seed=80 + s, layer=li).items()}
            packed = {k: torch.full_like(x[k], float("nan")) for k in ("q", "k_new", "v_new")}
            for k in packed:
                packed[k][:len(rows)] = x[k][rows]
            q_hat = g3.paged_append(packed["k_new"], packed["v_new"], gains[li][1], got["positions"], got["slots"], pool.k[li], pool.v[li],
                                    base, interp, q=packed["q"], q_gamma=gains[li][0])
            q_seq = newest_rows(q_hat, got["cu_tokens"])
            out, lse = g3.paged_decode(q_seq, pool.k[li], pool.v[li], pool.table, pool.lens, kind, win, return_lse=True)
            kept = [[c[waiting].clone() for c in pair] for pair in ring]
            lens = pool.lens.tolist()
            ref = g3.decode(x["q"], x["k_new"], x["v_new"], *gains[li], *ring[li], gi(lens), cap, kind, win, base, interp)
            for pair, old in zip(ring, kept):  # the contiguous call steps every sequence
                for c, o in zip(pair, old):
                    c[waiting] = o
            if rows:
                near(out[rows], ref[rows])
            if li == 1:
                g3.page_bounds(pool.k[1], pool.table, pool.old, pool.lens, pool.bounds, pool.exps)
                some = g3.page_select(q_seq, pool.bounds, pool.exps, pool.table, pool.lens, P, 2)
                part = g3.paged_decode(q_seq, pool.k[1], pool.v[1], pool.table, pool.lens, kind, win, pages=some)
                kp, vp = torch.nan_to_num(pool.k[1]).double().cpu().numpy(), torch.nan_to_num(pool.v[1]).double().cpu().numpy()
                if rows:
                    r = PG.paged_decode(q_seq[rows].cpu(), kp, vp, pool.table[rows].cpu(), pool.lens[rows].tolist(), 1, win, some[rows].cpu().numpy())
                    near(part[rows], torch.from_numpy(r[0]).to(dev()))
        assert torch.equal(pool.table[waiting], before[0][waiting]) and torch.equal(pool.lens[waiting], before[1][waiting])
        assert torch.equal(pool.bounds[theirs], before[2][theirs]) and torch.equal(pool.exps[theirs], before[3][theirs])
        for now, was in zip(pool.k + pool.v, before[4]):
            assert torch.equal(now[theirs].view(torch.int16), was[theirs].view(torch.int16))
        assert clean()


def test_captured_steps_with_waiting_sequences():
    """One captured step serves every choice of sequences that wait: the gather of the rows is in the graph."""
    def step(s):
        p = s.pool
        got = g3.page_map(p.lens, s.one, p.table, p.ring, p.state, p.P, p.n_pages, len(s.one))
        q_hat = g3.paged_append(s.k, s.v, s.gain, got["positions"], got["slots"], p.k[0], p.v[0], 1e6, 8.0, q=s.q, q_gamma=s.gain)
        g3.page_bounds(p.k[0], p.table, p.lens, got["seq_lens"], p.bounds, p.exps)
        q_seq = newest_rows(q_hat, got["cu_tokens"])
        pages = g3.page_select(q_seq, p.bounds, p.exps, p.table, got["seq_lens"], p.P, s.n)
        out, lse = g3.paged_decode(q_seq, p.k[0], p.v[0], p.table, got["seq_lens"], g3.GLOBAL, 0, pages=pages, return_lse=True)
        for into, new in ((s.out, out), (s.seen, lse), (p.lens, got["seq_lens"]), (p.state, got["free_state"])):
            into.copy_(new)
        return q_hat

    g3.paged_status(dev())
    eager, captured = Step(8), Step(8)
    for s in (eager, captured):
        step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    for active in ([1, 0, 1, 1, 0], [0, 0, 0, 0, 1], [1, 1, 1, 1, 1], [0, 0, 0, 0, 0], [0, 1, 0, 1, 0]) * 4:
        for s in (eager, captured):
            s.one.copy_(gi(active))
        q_hat, rows = step(eager), [b for b in range(5) if active[b]]
        graph.replay()
        torch.cuda.synchronize()
        same(eager, captured)
        if rows:  # each running sequence's output is the attention of its own packed row
            p, q = eager.pool, q_hat[:len(rows)].contiguous()
            table, lens = p.table[rows].contiguous(), p.lens[rows].contiguous()
            pages = g3.page_select(q, p.bounds, p.exps, table, lens, p.P, eager.n)
            near(eager.out[rows], g3.paged_decode(q, p.k[0], p.v[0], table, lens, g3.GLOBAL, 0, pages=pages))
    assert clean()


def test_a_step_runs_alike_without_the_quick_module(monkeypatch):
    """The calls of a box that built the C library alone: the ordinary way, the same bits."""
    a, b = Step(7), Step(7)
    for _ in range(3):
        a.run()
    monkeypatch.setattr(g3, "_quick", None)
    monkeypatch.setattr(g3, "HERE", "/nonexistent")
    with pytest.warns(RuntimeWarning, match="_paged.so is missing"):
        b.run()
    for _ in range(2):
        b.run()
    torch.cuda.synchronize()
    same(a, b)
    assert clean() and g3._quick is g3._Ordinary
