"""Pins of the paged-cache oracle: closed forms, the contiguous decode oracle, brute force."""
import math

import numpy as np
import pytest
import torch

import inputs
from oracle import attention as O
from oracle import paged as PG


def test_map_hands_out_pages_in_order_and_refuses_what_does_not_fit():
    table = np.full((4, 4), -1)
    table[0, :2] = [7, 3]
    ring = [11, 12, 13, 14, 10]
    got = PG.page_map([20, 0, 5, 0], [13, 16, 0, 40], table, ring, [4, 3], 16, 20, 100)
    # sequence 0: tokens 20..32 need one page (ring position 4 -> page 10); sequence 1 takes 11; 2 waits; 3 wants three, one is left
    assert got["table"][0].tolist() == [7, 3, 10, -1] and got["table"][1, 0] == 11 and (got["table"][3] == -1).all()
    assert got["seq_lens"].tolist() == [33, 16, 5, 0] and got["cu_tokens"].tolist() == [0, 13, 29, 29, 69]
    assert got["slots"][:13].tolist() == [3 * 16 + r for r in range(4, 16)] + [160]
    assert got["slots"][13:29].tolist() == list(range(176, 192)) and (got["slots"][29:] == -1).all()
    assert got["free_state"].tolist() == [1, 1] and got["error"]


@pytest.mark.parametrize("amax,e", [(127.0, 0), (127.5, -1), (1.0, 6), (1.9921875, 5), (0.0, 50), (math.inf, -50), (2.0 ** -80, 50)])
def test_exponent(amax, e):
    assert PG.exponent(amax) == e


def test_bounds_hold_every_key_and_scores_every_product():
    rng = np.random.default_rng(0)
    for _ in range(20):
        keys = torch.from_numpy(rng.normal(size=(rng.integers(1, 17), 64)) * 2.0 ** rng.integers(-9, 9)).bfloat16().double().numpy()
        bounds, e = PG.page_bounds_of(keys)
        assert (keys <= np.ldexp(bounds[0], -e)).all() and (keys >= np.ldexp(bounds[1], -e)).all()
        assert (np.ldexp(bounds[0] - 1, -e) < keys.max(0)).all() and (np.ldexp(bounds[1] + 1, -e) > keys.min(0)).all()  # and no wider
        q = np.rint(rng.normal(size=(3, 64)) * 30)   # whole numbers up to 127 are kept by the rounding of q
        q[:, 0] = 127
        score = PG.page_scores(q, bounds[None], [e])[0]
        assert score >= (keys @ q.T).max()
        assert score == max(PG.page_scores(row[None], bounds[None], [e])[0] for row in q)


def test_pick_ties_and_short_sequences():
    assert PG.page_pick([1, 5, 5, 5, 0, -9], 3).tolist() == [1, 2, 5]
    assert PG.page_pick([1, 5], 4).tolist() == [0, 1, -1, -1]
    assert PG.page_pick([], 2).tolist() == [-1, -1]
    assert PG.page_pick([3, 2, 1], 1).tolist() == [2]


@pytest.mark.parametrize("kind", [O.LOCAL, O.GLOBAL])
def test_paged_decode_equals_contiguous_decode(kind):
    B, Hq, Hkv, D, P, W = 2, 4, 2, 64, 16, 40
    lens, rng = [70, 33], np.random.default_rng(1)
    x = inputs.decode_step_inputs(B, Hq, Hkv, D, seed=1)
    base, interp = 1e4, 2.0
    hist, starts = [], []
    k_pages, v_pages = np.full((12, Hkv, P, D), np.nan), np.full((12, Hkv, P, D), np.nan)
    table = np.full((B, 5), -1)
    perm = rng.permutation(12)
    for b, L in enumerate(lens):
        t0 = max(0, L - W) if kind == O.LOCAL else 0
        h = inputs.cache_history(L - 1 - t0, Hkv, D, seed=2, layer=0, batch=b)
        hist.append(h)
        starts.append(t0)
        k_new = PG.norm_rope(x["k_new"][b][None], x["k_gamma"], [L - 1], base, interp)
        keys = np.concatenate([h["k"].double().numpy(), k_new])
        vals = np.concatenate([h["v"].double().numpy(), x["v_new"][b][None].double().numpy()])
        for i, t in enumerate(range(t0, L)):
            table[b, t // P] = perm[b * 6 + t // P]
            k_pages[table[b, t // P], :, t % P], v_pages[table[b, t // P], :, t % P] = keys[i], vals[i]
    q_hat = np.stack([PG.norm_rope(x["q"][b][None], x["q_gamma"], [L - 1], base, interp)[0] for b, L in enumerate(lens)])
    out, lse, _, _ = PG.paged_decode(q_hat, k_pages, v_pages, table, lens, kind, W)
    ref, _ = O.decode(x["q"], x["k_new"], x["v_new"], x["q_gamma"], x["k_gamma"], lens, [h["k"] for h in hist],
                      [h["v"] for h in hist], starts, kind, W, base, interp)
    np.testing.assert_allclose(out, ref, rtol=1e-12, atol=1e-13)
    assert np.isfinite(lse).all()
    if kind == O.GLOBAL:  # a list of all pages is the same; the newest page alone sees its own tokens only
        every = np.where(np.arange(5) < -(-np.array(lens) // P)[:, None], np.arange(5), -1)[:, None].repeat(Hkv, 1)
        np.testing.assert_array_equal(PG.paged_decode(q_hat, k_pages, v_pages, table, lens, kind, W, every)[0], out)
        one = PG.paged_decode(q_hat, k_pages, v_pages, table, lens, kind, W, np.full((B, Hkv, 1), 2))
        assert np.isfinite(one[0]).all() and (one[1] < lse).all()
