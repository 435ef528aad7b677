"""The paged calls as a server uses them: prompts and decode steps over a block of layers, captured steps, streams,
the binding's two ways and its refusals.

The reference of a decode step is g3attn_decode on contiguous caches (itself checked against the float64 oracle within
ATOL / REL_L2 of the outputs); the paged step rounds q_hat to bf16 where that one keeps fp32, so the bar is those two
tolerances added."""
import numpy as np
import pytest
import torch

import global_gqa_b200 as g3
import inputs
from oracle import paged as PG
from gpu_helpers import ATOL, REL_L2, dev

pytestmark = pytest.mark.gpu
i32 = torch.int32


def gi(x):
    return torch.as_tensor(np.asarray(x), dtype=i32).to(dev())


def near(a, b):
    d, r = (a.double() - b.double()).cpu().numpy(), b.double().cpu().numpy()
    assert np.isfinite(d).all() and np.abs(d).max() <= 2 * ATOL and np.linalg.norm(d) <= 2 * REL_L2 * np.linalg.norm(r)


class Pool:
    """Pages, bounds and the free ring of a server's layers; the block table and lengths of its sequences."""

    def __init__(self, layers, n_pages, B, max_pages, Hkv, D, P, seed=0):
        z = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device=dev())  # noqa: E731
        self.k, self.v = ([z(n_pages, Hkv, P, D) for _ in range(layers)] for _ in "kv")
        self.bounds = torch.zeros(n_pages, Hkv, 2, D, dtype=torch.int8, device=dev())
        self.exps = torch.zeros(n_pages, Hkv, dtype=torch.int8, device=dev())
        self.table = torch.full((B, max_pages), -1, dtype=i32, device=dev())
        self.ring = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(i32).to(dev())
        self.state = gi([0, n_pages])
        self.lens = gi([0] * B)
        self.P, self.n_pages = P, n_pages

    def map(self, new, T):
        """One step's slots: lengths and ring move on."""
        got = g3.page_map(self.lens, gi(new), self.table, self.ring, self.state, self.P, self.n_pages, T)
        self.old, self.lens, self.state = self.lens, got["seq_lens"], got["free_state"]
        return got

    def give_back(self, b):
        """A finished sequence's pages go behind the ring's last one."""
        n = -(-int(self.lens[b]) // self.P)
        head, count = self.state.tolist()
        at = (head + count + torch.arange(n, device=dev())) % self.ring.numel()
        self.ring[at] = self.table[b, :n]
        self.state = gi([head, count + n])
        self.lens = self.lens.clone()
        self.lens[b] = 0


def layer(li, W):
    return (g3.LOCAL, W, 1e4, 1.0) if li == 0 else (g3.GLOBAL, W, 1e6, 8.0)


@pytest.mark.parametrize("Hq,Hkv,D,P", [(4, 2, 64, 16), (8, 2, 128, 32), (4, 1, 256, 16)])
def test_prompts_then_decode_steps(Hq, Hkv, D, P):
    """Prompts of different lengths, a sequence that joins later, one that ends and whose pages are taken again."""
    B, W, cap = 4, 48, 400
    prompts = [70, 0, 200, 33]
    pool = Pool(2, 40, B, -(-cap // P), Hkv, D, P)
    ring = [[torch.zeros(B, Hkv, W if li == 0 else cap, D, dtype=torch.bfloat16, device=dev()) for _ in "kv"] for li in range(2)]
    gains = [inputs.prefill_layer_inputs(1, 1, Hq, Hkv, D, seed=0, layer=li) for li in range(2)]
    gains = [(x["q_gamma"].to(dev()), x["k_gamma"].to(dev())) for x in gains]

    def prompt(b, n, seed, packed, got, li):
        """Prefill of sequence b into its contiguous cache, and the same tokens into the pages."""
        kind, win, base, interp = layer(li, W)
        x = inputs.prefill_layer_inputs(1, n, Hq, Hkv, D, seed=seed, layer=li)
        x = {k: v.to(dev()) for k, v in x.items() if v is not None}
        qg, kg = gains[li]
        kc, vc = (torch.zeros(1, Hkv, W if li == 0 else cap, D, dtype=torch.bfloat16, device=dev()) for _ in "kv")
        g3.prefill(x["q"], x["k"], x["v"], qg, kg, x["positions"], kind, win, base, interp, k_cache=kc, v_cache=vc)
        ring[li][0][b], ring[li][1][b] = kc[0], vc[0]
        r0 = int(got["cu_tokens"][b])
        packed[0][r0:r0 + n], packed[1][r0:r0 + n] = x["k"][0], x["v"][0]

    def feed(new, seeds):
        T = sum(new) + 5  # a padded batch
        got = pool.map(new, T)
        for li in range(2):
            kind, win, base, interp = layer(li, W)
            packed = [torch.full((T, Hkv, D), float("nan"), dtype=torch.bfloat16, device=dev()) for _ in "kv"]
            for b, n in enumerate(new):
                if n:
                    prompt(b, n, seeds[b], packed, got, li)
            assert g3.paged_append(packed[0], packed[1], gains[li][1], got["positions"], got["slots"], pool.k[li], pool.v[li],
                                   base, interp) is None
        g3.page_bounds(pool.k[1], pool.table, pool.old, pool.lens, pool.bounds, pool.exps)

    def step(active, seed):
        got = pool.map([int(a) for a in active], B)
        rows = [b for b in range(B) if active[b]]
        x = [inputs.decode_step_inputs(B, Hq, Hkv, D, seed=seed, layer=li) for li in range(2)]
        for li in range(2):
            kind, win, base, interp = layer(li, W)
            qg, kg = gains[li]
            xd = {k: v.to(dev()) for k, v in x[li].items()}
            packed = {k: torch.zeros_like(xd[k]) for k in ("q", "k_new", "v_new")}
            for k in packed:
                packed[k][:len(rows)] = xd[k][rows]
            q_hat = g3.paged_append(packed["k_new"], packed["v_new"], kg, got["positions"], got["slots"], pool.k[li], pool.v[li],
                                    base, interp, q=packed["q"], q_gamma=qg)
            q_seq = torch.zeros_like(q_hat)
            q_seq[rows] = q_hat[:len(rows)]
            out, lse = g3.paged_decode(q_seq, pool.k[li], pool.v[li], pool.table, pool.lens, kind, win, return_lse=True)
            lens = pool.lens.tolist()
            ref = g3.decode(xd["q"], xd["k_new"], xd["v_new"], qg, kg, *ring[li], gi([max(n, 1) for n in lens]), cap, kind, win,
                            base, interp)
            idle = [b for b in range(B) if lens[b] == 0]
            assert (out[idle] == 0).all() and (lse[idle] == -float("inf")).all()
            near(out[rows], ref[rows])
            for b in idle:  # the contiguous call takes no idle sequence: what it wrote there goes
                ring[li][0][b] = ring[li][1][b] = 0
            if li == 1:
                g3.page_bounds(pool.k[1], pool.table, pool.old, pool.lens, pool.bounds, pool.exps)
                every = g3.page_select(q_seq, pool.bounds, pool.exps, pool.table, pool.lens, P, pool.table.shape[1])
                got_all = g3.paged_decode(q_seq, pool.k[1], pool.v[1], pool.table, pool.lens, kind, win, pages=every, return_lse=True)
                near(got_all[0][rows], out[rows])  # all pages selected: the same tokens, cut in other places
                assert ((got_all[1] - lse)[rows].abs() < 1e-4).all()
                some = g3.page_select(q_seq, pool.bounds, pool.exps, pool.table, pool.lens, P, 3)
                part, part_lse = g3.paged_decode(q_seq, pool.k[1], pool.v[1], pool.table, pool.lens, kind, win, pages=some, return_lse=True)
                kp, vp = torch.nan_to_num(pool.k[1]).double().cpu().numpy(), torch.nan_to_num(pool.v[1]).double().cpu().numpy()
                r, rl, _, _ = PG.paged_decode(q_seq.cpu(), kp, vp, pool.table.cpu(), lens, 1, win, some.cpu().numpy())
                near(part[rows], torch.from_numpy(r)[rows].to(dev()))
                assert (part_lse[rows] <= lse[rows] + 1e-4).all()

    feed(prompts, [11, 0, 12, 13])
    for s in range(3):
        step([True, False, True, True], 20 + s)
    feed([0, 90, 0, 0], [0, 14, 0, 0])
    for s in range(3):
        step([True] * 4, 30 + s)
    pool.give_back(2)
    feed([0, 0, 120, 0], [0, 0, 15, 0])
    for s in range(20):
        step([True, s % 2 == 0, True, s < 4], 40 + s) if s % 2 == 0 and s < 4 else step([True] * 4, 40 + s)
    assert g3.check_device_error(g3.paged_status(dev())) == 0
    taken = pool.table[pool.table >= 0]
    assert int(pool.state[1]) + sum(-(-n // P) for n in pool.lens.tolist()) == pool.n_pages
    live = torch.cat([pool.table[b, :-(-int(n) // P)] for b, n in enumerate(pool.lens.tolist())])
    assert live.unique().numel() == live.numel() and taken.max() < pool.n_pages  # no page belongs to two sequences


class Step:
    """One captured decode step of a sparse global layer: map, append, bounds, selection, attention; lengths move on in place."""

    def __init__(self, seed, B=5, Hq=8, Hkv=2, D=128, P=16, n=4):
        self.pool = pool = Pool(1, 60 * B, B, 50, Hkv, D, P, seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.gain = torch.ones(D, device=dev())
        lens = [40 * b + 3 for b in range(B)]
        got = pool.map(lens, sum(lens))
        g3.paged_append(r(sum(lens), Hkv, D), r(sum(lens), Hkv, D), self.gain, got["positions"], got["slots"], pool.k[0], pool.v[0], 1e6, 8.0)
        g3.page_bounds(pool.k[0], pool.table, pool.old, pool.lens, pool.bounds, pool.exps)
        self.q, self.k, self.v, self.one = r(B, Hq, D), r(B, Hkv, D), r(B, Hkv, D), gi([1] * B)
        self.n = n
        self.out = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=dev())
        self.seen = torch.zeros(B, Hq, dtype=torch.float32, device=dev())

    def run(self):
        p = self.pool
        got = g3.page_map(p.lens, self.one, p.table, p.ring, p.state, p.P, p.n_pages, len(self.one))
        q_hat = g3.paged_append(self.k, self.v, self.gain, got["positions"], got["slots"], p.k[0], p.v[0], 1e6, 8.0, q=self.q,
                                q_gamma=self.gain)
        g3.page_bounds(p.k[0], p.table, p.lens, got["seq_lens"], p.bounds, p.exps)
        pages = g3.page_select(q_hat, p.bounds, p.exps, p.table, got["seq_lens"], p.P, self.n)
        out, lse = g3.paged_decode(q_hat, p.k[0], p.v[0], p.table, got["seq_lens"], g3.GLOBAL, 0, pages=pages, return_lse=True)
        self.out.copy_(out)
        self.seen.copy_(lse)
        p.lens.copy_(got["seq_lens"])
        p.state.copy_(got["free_state"])
        # inputs of the next step follow from this one's output
        self.q.copy_((self.q.float() * 0.5 + out.float()).bfloat16())
        self.k.copy_(out[:, ::4] * 2)


def same(a, b):
    for x, y in ((a.out, b.out), (a.seen, b.seen), (a.pool.lens, b.pool.lens), (a.pool.table, b.pool.table), (a.pool.state, b.pool.state),
                 (a.pool.bounds, b.pool.bounds)):
        assert torch.equal(x, y)


def test_captured_steps_and_two_graphs_at_once():
    """Steps replayed from a graph, and two graphs captured on one stream replayed side by side, as eager ones run."""
    g3.paged_status(dev())
    eager = [Step(s) for s in (1, 2)]
    for e in eager:
        for _ in range(30):
            e.run()
    steps, graphs, streams = [Step(s) for s in (1, 2)], [], [torch.cuda.Stream() for _ in range(2)]
    for s in steps:
        s.run()  # the call before a capture
    torch.cuda.synchronize()
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for _ in range(29):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, steps):
        assert torch.isfinite(a.out.float()).all()
        same(a, b)
    assert g3.check_device_error(g3.paged_status(dev())) == 0


def test_own_status_in_a_capture_and_bad_lengths_from_a_replay():
    s = Step(3)
    status = torch.zeros(2, dtype=i32, device=dev())
    q_hat = torch.randn(5, 8, 128, device=dev()).bfloat16()
    lens, p = s.pool.lens.clone(), s.pool
    g3.paged_decode(q_hat, p.k[0], p.v[0], p.table, lens, g3.GLOBAL, 0, status=status)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = g3.paged_decode(q_hat, p.k[0], p.v[0], p.table, lens, g3.GLOBAL, 0, status=status)
    g.replay()
    assert g3.check_device_error(status) == 0 and (out[1:] != 0).any()
    lens[2] = -1
    g.replay()
    assert g3.check_device_error(status) == 1 and (out[2] == 0).all()
    assert g3.check_device_error(status) == 0
    assert g3.check_device_error(g3.paged_status(dev())) == 0  # the device's own words hold nothing of it


def test_streams_and_both_ways_of_the_binding_agree():
    """The ordinary way (given outputs, another stream) and the quick one give the same bits; two streams at once."""
    a, b = Step(4), Step(4)
    a.run()
    p = b.pool
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n, B = len(b.one), 5
    outs = {k: torch.empty(m, dtype=i32, device=dev()) for k, m in (("seq_lens", n), ("cu_tokens", n + 1), ("slots", n), ("positions", n),
                                                                  ("free_state", 2))}
    got = g3.page_map(p.lens, b.one, p.table, p.ring, p.state, p.P, p.n_pages, n, out=outs, stream=side)
    assert all(got[k] is outs[k] for k in outs)
    q_hat = torch.empty_like(b.q)
    back = g3.paged_append(b.k, b.v, b.gain, got["positions"], got["slots"], p.k[0], p.v[0], 1e6, 8.0, q=b.q, q_gamma=b.gain, q_hat=q_hat,
                           stream=side)
    assert back is q_hat
    g3.page_bounds(p.k[0], p.table, p.lens, got["seq_lens"], p.bounds, p.exps, stream=side)
    ws = torch.empty(g3.page_select_workspace_size(B, 2, 50), dtype=torch.uint8, device=dev())
    pages = g3.page_select(q_hat, p.bounds, p.exps, p.table, got["seq_lens"], p.P, b.n, ws=ws, stream=side)
    ws = torch.empty(g3.paged_decode_workspace_size(128), dtype=torch.uint8, device=dev())
    out, lse = g3.paged_decode(q_hat, p.k[0], p.v[0], p.table, got["seq_lens"], g3.GLOBAL, 0, pages=pages, return_lse=True, ws=ws,
                               out=b.out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, a.out) and torch.equal(lse, a.seen) and torch.equal(got["seq_lens"], a.pool.lens)
    assert torch.equal(p.table, a.pool.table) and torch.equal(p.bounds, a.pool.bounds)
    # many calls on two streams, each with outputs and workspaces of its own
    want = [g3.paged_decode(q_hat * s, p.k[0], p.v[0], p.table, got["seq_lens"], g3.GLOBAL, 0) for s in (1, 2)]
    torch.cuda.synchronize()
    lanes, results = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(20):
        for s, st in zip((1, 2), lanes):
            with torch.cuda.stream(st):
                results.append((s, g3.paged_decode(q_hat * s, p.k[0], p.v[0], p.table, got["seq_lens"], g3.GLOBAL, 0)))
    torch.cuda.synchronize()
    assert all(torch.equal(r, want[s - 1]) for s, r in results)


def test_binding_refuses_before_anything_runs():
    s = Step(6)
    p, q = s.pool, s.q
    dec = dict(q_hat=q, k_pages=p.k[0], v_pages=p.v[0], block_table=p.table, seq_lens=p.lens, layer_kind=g3.GLOBAL, window=0)
    good = g3.paged_decode(**dec)

    def refused(fn, args, error, match, **kw):
        with pytest.raises(error, match=match):
            fn(**{**args, **kw})

    refused(g3.paged_decode, dec, TypeError, "q_hat must be", q_hat=q.float())
    refused(g3.paged_decode, dec, ValueError, "contiguous", q_hat=q.transpose(0, 1))
    refused(g3.paged_decode, dec, ValueError, "v_pages must have shape", v_pages=p.v[0][:-1])
    refused(g3.paged_decode, dec, TypeError, "block_table must be", block_table=p.table.long())
    refused(g3.paged_decode, dec, ValueError, "seq_lens must", seq_lens=p.lens[:-1])
    refused(g3.paged_decode, dec, ValueError, "CUDA", seq_lens=p.lens.cpu())
    refused(g3.paged_decode, dec, ValueError, "status must", status=torch.zeros(3, dtype=i32, device=dev()))
    refused(g3.paged_decode, dec, ValueError, "out must", out=q[:2])
    refused(g3.paged_decode, dec, g3.G3Error, "window", layer_kind=g3.LOCAL)
    refused(g3.paged_decode, dec, g3.G3Error, "bad layer kind", layer_kind=5)
    refused(g3.paged_decode, dec, ValueError, "32 bits", layer_kind=g3.LOCAL, window=2 ** 32 + 5)
    refused(g3.paged_decode, dec, g3.G3Error, "workspace", ws=torch.empty(64, dtype=torch.uint8, device=dev()))
    refused(g3.paged_decode, dec, g3.G3Error, "page list is for global", pages=gi(np.zeros((5, 2, 3))), layer_kind=g3.LOCAL, window=4)
    refused(g3.paged_decode, dec, ValueError, "no entries", pages=gi(np.zeros((5, 2, 0))))
    refused(g3.paged_decode, dec, ValueError, "pages must have shape", pages=gi(np.zeros((5, 3, 3))))
    sel = dict(q_hat=q, bounds=p.bounds, exps=p.exps, block_table=p.table, seq_lens=p.lens, page_size=16, n_select=3)
    refused(g3.page_select, sel, g3.G3Error, "n_select", n_select=0)
    refused(g3.page_select, sel, g3.G3Error, "page_size", page_size=20)
    refused(g3.page_select, sel, ValueError, "32 bits", n_select=2 ** 32 + 3)
    refused(g3.page_select, sel, ValueError, "32 bits", page_size=2 ** 32 + 16)
    refused(g3.page_select, sel, TypeError, "bounds must be", bounds=p.bounds.to(torch.uint8))
    app = dict(k=s.k, v=s.v, k_gamma=s.gain, positions=s.one, slots=s.one, k_pages=p.k[0], v_pages=p.v[0], rope_base=1e4, interp_factor=1.0)
    refused(g3.paged_append, app, ValueError, "q_gamma and q_hat", q_gamma=s.gain)
    refused(g3.paged_append, app, TypeError, "q_gamma must", q=q)
    refused(g3.paged_append, app, g3.G3Error, "rope_base", rope_base=-1.0)
    refused(g3.paged_append, app, ValueError, "positions must have shape", positions=s.one[:2])
    mp = dict(old_lens=p.lens, new_lens=s.one, block_table=p.table, free_pages=p.ring, free_state=p.state, page_size=16, n_pages=p.n_pages,
              max_tokens=5)
    refused(g3.page_map, mp, g3.G3Error, "overlaps", out=dict(seq_lens=p.lens))
    refused(g3.page_map, mp, g3.G3Error, "max_tokens", max_tokens=0)
    refused(g3.page_map, mp, ValueError, "32 bits", max_tokens=2 ** 32 + 5)
    refused(g3.page_map, mp, ValueError, "32 bits", n_pages=2 ** 32 + 5)
    refused(g3.page_map, mp, ValueError, "free_state must have shape", free_state=p.lens)
    bd = dict(k_pages=p.k[0], block_table=p.table, old_lens=p.lens, seq_lens=p.lens, bounds=p.bounds, exps=p.exps)
    refused(g3.page_bounds, bd, ValueError, "exps must have shape", exps=p.exps[:, :1].contiguous())
    assert torch.equal(g3.paged_decode(**dec), good) and g3.check_device_error(g3.paged_status(dev())) == 0
