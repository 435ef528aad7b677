"""Host-side refusals of the paged-cache calls: nothing is launched, no GPU is needed."""
import os

import pytest

import global_gqa_b200 as g3

FAKE = 0x100000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(g3.LIB_PATH) or not os.path.exists(os.path.join(g3.HERE, "_paged.so")):
        from global_gqa_b200 import build
        build.build()
    return g3.lib()


def at(i):
    return FAKE + i * 0x100000


CALLS = {
    "g3attn_page_map": dict(old=at(0), new=at(1), B=4, table=at(2), max_pages=8, free=at(3), cap=64, state=at(4), P=16,
                            n_pages=64, T=100, lens=at(5), cu=at(6), slots=at(7), pos=at(8), state_out=at(9),
                            status=None, stream=None),
    "g3attn_paged_append": dict(q=at(0), k=at(1), v=at(2), qg=at(3), kg=at(4), pos=at(5), slots=at(6), kp=at(7), vp=at(8),
                                n_pages=10, P=64, base=1e4, interp=1.0, T=5, Hq=4, Hkv=2, D=128, qh=at(9), status=None,
                                stream=None),
    "g3attn_page_bounds": dict(kp=at(0), table=at(1), old=at(2), lens=at(3), B=2, max_pages=4, n_pages=10, P=64, Hkv=2,
                               D=128, bounds=at(4), exps=at(5), status=None, stream=None),
    "g3attn_page_select": dict(qh=at(0), bounds=at(1), exps=at(2), table=at(3), lens=at(4), B=2, max_pages=4, n_pages=10,
                               P=64, Hq=4, Hkv=2, D=128, n=2, pages=at(5), ws=at(6), wsb=1 << 30, status=None,
                               stream=None),
    "g3attn_paged_decode": dict(qh=at(0), kp=at(1), vp=at(2), table=at(3), lens=at(4), pages=None, n=0, kind=1, window=0,
                                B=2, max_pages=4, n_pages=10, P=64, Hq=4, Hkv=2, D=128, out=at(5), lse=None, ws=at(6),
                                wsb=1 << 30, status=None, stream=None),
}

REFUSED = [
    ("page_map", dict(old=None), 1), ("page_map", dict(state_out=None), 1), ("page_map", dict(B=0), 1),
    ("page_map", dict(T=0), 1), ("page_map", dict(cap=0), 1), ("page_map", dict(n_pages=0), 1), ("page_map", dict(P=24), 2),
    ("page_map", dict(P=512), 2), ("page_map", dict(B=8193), 2), ("page_map", dict(n_pages=1 << 28), 2),
    ("page_map", dict(B=8192, max_pages=1 << 18), 2), ("page_map", dict(T=(1 << 30) + 1), 2),
    ("page_bounds", dict(B=64, Hkv=16, max_pages=1 << 18), 2), ("paged_decode", dict(B=64, Hq=16, Hkv=16, max_pages=1 << 18), 2), ("page_map", dict(lens=at(0)), 1),      # in place over an input
    ("page_map", dict(state_out=at(4) + 4), 1), ("page_map", dict(slots=at(8) - 100), 1),     # half over another output
    ("page_map", dict(table=at(3) - 4), 1),
    ("page_map", dict(B=1, max_pages=(1 << 27) - 1), 2), ("page_bounds", dict(B=1, P=256, max_pages=(1 << 23) - 1), 2),
    ("paged_append", dict(k=None), 1), ("paged_append", dict(T=-1), 1), ("paged_append", dict(base=0.0), 1),
    ("paged_append", dict(base=float("nan")), 1), ("paged_append", dict(interp=float("inf")), 1),
    ("paged_append", dict(Hq=0), 1), ("paged_append", dict(q=None), 1), ("paged_append", dict(qh=None), 1),
    ("paged_append", dict(Hkv=0), 1), ("paged_append", dict(D=0), 1), ("paged_append", dict(D=96), 2),
    ("paged_append", dict(P=8), 2), ("paged_append", dict(v=at(2) + 8), 1), ("paged_append", dict(kp=at(7) + 2), 1),
    ("page_bounds", dict(exps=None), 1), ("page_bounds", dict(B=0), 1), ("page_bounds", dict(D=512), 2),
    ("page_bounds", dict(kp=at(0) + 8), 1), ("page_bounds", dict(max_pages=0), 1), ("page_bounds", dict(P=17), 2),
    ("page_select", dict(pages=None), 1), ("page_select", dict(n=0), 1), ("page_select", dict(Hq=5), 1),
    ("page_select", dict(Hq=18), 2), ("page_select", dict(ws=None), 3), ("page_select", dict(wsb=16), 3),
    ("page_select", dict(ws=at(6) + 16), 3), ("page_select", dict(qh=at(0) + 2), 1),
    ("paged_decode", dict(qh=None), 1), ("paged_decode", dict(kind=2), 1), ("paged_decode", dict(kind=0, window=0), 1),
    ("paged_decode", dict(pages=at(7)), 1), ("paged_decode", dict(n=3), 1), ("paged_decode", dict(n=-1, pages=at(7)), 1),
    ("paged_decode", dict(pages=at(7), n=2, kind=0, window=5), 2), ("paged_decode", dict(Hq=3), 1),
    ("paged_decode", dict(Hq=18), 2), ("paged_decode", dict(D=32), 2), ("paged_decode", dict(B=9000), 2),
    ("paged_decode", dict(ws=None), 3), ("paged_decode", dict(wsb=1000), 3), ("paged_decode", dict(ws=at(6) + 64), 3),
    ("paged_decode", dict(vp=at(2) + 4), 1), ("paged_decode", dict(out=at(5) + 8), 1),
]


@pytest.mark.parametrize("call,kw,code", REFUSED, ids=[f"{c}-{'-'.join(k)}-{i}" for i, (c, k, _) in enumerate(REFUSED)])
def test_refused_on_host(lib, call, kw, code):
    a = dict(CALLS["g3attn_" + call])
    assert set(kw) <= set(a)
    a.update(kw)
    assert getattr(lib, "g3attn_" + call)(*a.values()) == code
    assert lib.g3attn_last_error().startswith(call.encode())


def test_no_tokens_is_no_work(lib):
    a = dict(CALLS["g3attn_paged_append"], T=0, q=None, k=None, qg=None, qh=None, Hq=0)
    assert lib.g3attn_paged_append(*a.values()) == 0


def test_workspace_sizes(lib):
    assert 0 < lib.g3attn_page_select_workspace_size(64, 16, 8192) <= 4096  # scores stay on chip
    assert lib.g3attn_page_select_workspace_size(64, 16, 8193) == 64 * 16 * 8193 * 4
    assert lib.g3attn_page_select_workspace_size(0, 16, 2048) == 0
    # two partial softmaxes per block, whatever the batch and the lengths
    assert lib.g3attn_paged_decode_workspace_size(96) == 0 and lib.g3attn_paged_decode_workspace_size(128) >= 2 * 148 * 8 * 128 * 4


def test_binding_refuses_cpu_tensors():
    import torch
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        g3.page_map(i32, i32, i32[:, None], i32, i32, 16, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        g3.paged_decode(torch.zeros(2, 4, 64, dtype=torch.bfloat16), None, None, None, None, g3.GLOBAL, 0)
