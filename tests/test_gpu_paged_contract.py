"""What the paged calls' documentation promises at the edges of their arguments, one promise per test.

Tolerances are those that test_gpu_paged.py derives."""
import numpy as np
import pytest
import torch

import global_gqa_b200 as g3
from oracle import paged as PG
from gpu_helpers import dev
from test_gpu_paged import check_select, clean, decode_case, gi, near_decode
from test_gpu_paged_serving import Step, same

pytestmark = pytest.mark.gpu


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
