"""The paged-cache oracle's pins must catch plausible mistakes: each case plants one and requires a pin to fail."""
import inspect
import math

import numpy as np
import pytest

from oracle import paged as PG
import test_oracle_paged as PINS

# (function, its text, the mistaken text)
MUTANTS = {
    "map_pages_rounded_down": ("page_map", "-(-(old + new) // P)", "(old + new) // P"),
    "map_ring_not_wrapped": ("page_map", "(head + asked - total + j) % cap", "min(head + asked - total + j, cap - 1)"),
    "map_refused_loses_its_rows": ("page_map", "row0, row = row, row + max(new, 0)", "row0, row = row, row + (max(new, 0) if new < 40 else 0)"),
    "map_grants_past_the_ring": ("page_map", "granted = total == have or asked <= count", "granted = True"),
    "map_slot_by_token_not_row": ("page_map", "page * P + (old + i) % P", "page * P + i % P"),
    "exponent_one_too_high": ("exponent", "math.ldexp(amax, e) > 127", "math.ldexp(amax, e) > 254"),
    "bounds_inward": ("page_bounds_of", "np.floor(np.ldexp(small, e))", "np.ceil(np.ldexp(small, e))"),
    "bounds_largest_by_size": ("page_bounds_of", "rows.max(0), rows.min(0)", "np.abs(rows).max(0), rows.min(0)"),
    "score_swaps_the_bounds": ("page_scores", "np.minimum(q8, 0) @ _f64(bounds)[:, 1].T", "np.minimum(q8, 0) @ _f64(bounds)[:, 0].T"),
    "score_of_the_first_head": ("page_scores", "best = np.maximum(best,", "best = best if best[0] > -math.inf else np.maximum(best,"),
    "pick_ties_to_the_last": ("page_pick", "(-scores[j], j)", "(-scores[j], -j)"),
    "pick_forgets_the_newest": ("page_pick", "got = sorted(others) + [n - 1]", "got = sorted(others)"),
    "decode_window_off_by_one": ("paged_decode", "max(0, L - window)", "max(0, L - window - 1)"),
    "decode_whole_last_page": ("paged_decode", "(toks < L)", "(toks < L + 1)"),
    "decode_heads_by_modulo": ("paged_decode", "range(h * G, (h + 1) * G)", "range(h, Hq, Hkv)"),
    "decode_no_scale": ("paged_decode", "K @ q[b, g] / math.sqrt(D)", "K @ q[b, g]"),
}


def pins_caught():
    caught = []
    for name, f in sorted(vars(PINS).items()):
        if not name.startswith("test_"):
            continue
        cases = [()]
        for mark in getattr(f, "pytestmark", []):
            if mark.name == "parametrize":
                cases = [c if isinstance(c, tuple) else (c,) for c in mark.args[1]]
        for c in cases:
            try:
                f(*c)
            except (AssertionError, IndexError, ValueError):
                caught.append(name)
    return caught


def test_pins_pass_on_the_oracle_itself():
    assert pins_caught() == []


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_pins_catch_mutant(name, monkeypatch):
    fn, text, wrong = MUTANTS[name]
    source = inspect.getsource(getattr(PG, fn))
    assert source.count(text) >= 1, text
    space = dict(vars(PG), np=np, math=math)
    exec(source.replace(text, wrong), space)
    monkeypatch.setattr(PG, fn, space[fn])
    assert pins_caught(), f"no pin caught mutant {name}"
