"""Python binding of libg3attn (Gemma 3 5:1 block attention on B200).

Argument marshalling only: every step of the computation runs in the CUDA
library behind the C ABI declared in include/g3attn.h.  torch supplies device
memory and the current stream.  There is no fallback: if the library is not
built or no CUDA device is present, the calls raise.
"""
from __future__ import annotations

import ctypes
import os
import re
import warnings
from typing import Optional, Tuple

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB_PATH = os.path.join(HERE, "libg3attn.so")
HEADER_PATH = os.path.join(ROOT, "include", "g3attn.h")

LOCAL = 0
GLOBAL = 1

STATUS = {0: "G3_OK", 1: "G3_ERR_INVALID_ARG", 2: "G3_ERR_UNSUPPORTED", 3: "G3_ERR_WORKSPACE",
          4: "G3_ERR_CUDA", 5: "G3_ERR_TIMEOUT"}


class G3Error(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}: {detail}")


class KernelTrace(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int64), ("total_ms", ctypes.c_double)]


_lib = None

_vp, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t

_SIGS = {
    "g3attn_prefill_workspace_size": (_sz, [_i32] * 5),
    "g3attn_prefill": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _i32, _f32, _f32, _vp, _i32,
                                      _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _sz, _vp]),
    "g3attn_prefill_chunk_workspace_size": (_sz, [_i32] * 6 + [ctypes.c_int, _i32]),
    "g3attn_prefill_chunk": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, ctypes.c_int, _i32,
                                            _f32, _f32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp,
                                            _sz, _vp]),
    "g3attn_prefill_backward_workspace_size": (_sz, [_i32] * 5),
    "g3attn_prefill_backward": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _i32, _f32, _f32, _vp,
                                               _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                               _vp, _vp, _vp, _sz, _vp]),
    "g3attn_soft_tokens": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp]),
    "g3attn_decode_workspace_size": (_sz, [_i32] * 5),
    "g3attn_decode": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, ctypes.c_int, _i32,
                                     _f32, _f32, _i32, _i32, _i32, _i32, _vp, _vp, _sz, _vp]),
    "g3attn_decode_no_alloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, ctypes.c_int,
                                              _i32, _f32, _f32, _i32, _i32, _i32, _i32, _vp, _vp]),
    "g3attn_page_map": (ctypes.c_int, [_vp, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                       _vp, _vp, _vp]),
    "g3attn_paged_append": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _f32, _f32, _i32,
                                           _i32, _i32, _i32, _vp, _vp, _vp]),
    "g3attn_page_bounds": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "g3attn_page_select_workspace_size": (_sz, [_i32] * 3),
    "g3attn_page_select": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp,
                                          _vp, _sz, _vp, _vp]),
    "g3attn_paged_decode_workspace_size": (_sz, [_i32]),
    "g3attn_paged_decode": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, ctypes.c_int, _i32, _i32, _i32, _i32,
                                           _i32, _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp, _vp]),
    "g3attn_check_device_error": (ctypes.c_int, [_vp, _vp]),
    "g3attn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "g3attn_last_error": (ctypes.c_char_p, []),
    "g3attn_trace_enable": (ctypes.c_int, [ctypes.c_int]),
    "g3attn_trace_collect": (_i32, [ctypes.POINTER(KernelTrace), _i32]),
}


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m global_gqa_b200.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib


def header_functions() -> list:
    """Names of the functions include/g3attn.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(g3attn_\w+)\s*\(", text)))


def _check(status: int, where: str) -> None:
    if status != 0:
        detail = lib().g3attn_last_error().decode(errors="replace")
        raise G3Error(status, where, detail)


def prefill_workspace_size(B: int, S: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().g3attn_prefill_workspace_size(B, S, Hq, Hkv, D))


def prefill_chunk_workspace_size(B: int, C: int, Hq: int, Hkv: int, D: int, start: int, layer_kind: int,
                                 window: int) -> int:
    return int(lib().g3attn_prefill_chunk_workspace_size(B, C, Hq, Hkv, D, start, int(layer_kind), window))


def prefill_backward_workspace_size(B: int, S: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().g3attn_prefill_backward_workspace_size(B, S, Hq, Hkv, D))


def decode_workspace_size(B: int, Hq: int, Hkv: int, D: int, max_seq_len: int) -> int:
    return int(lib().g3attn_decode_workspace_size(B, Hq, Hkv, D, max_seq_len))


# ----------------------------------------------------------- torch plumbing
def _torch():
    import torch
    return torch


_workspaces = {}


def workspace(nbytes: int, device, tag: str = "default", stream=None):
    """A cached uint8 device buffer of at least nbytes (256-byte aligned).

    One buffer per (device, tag, stream): calls on one stream run in order and
    may share it, calls on different streams may overlap and must not (stream
    None is the device's current stream, as in the calls).
    """
    torch = _torch()
    device = torch.device(device)
    if device.index is None:  # "cuda" means the current device: name it as tensors do
        device = torch.device("cuda", torch.cuda.current_device())
    s = stream if stream is not None else torch.cuda.current_stream(device)
    key = (str(device), tag, int(s.cuda_stream))
    buf = _workspaces.get(key)
    if buf is None or buf.numel() < nbytes:
        # Allocated on the stream that uses it, so that when a larger buffer
        # replaces it, torch reuses the old memory only after that stream's
        # earlier calls have finished with it.
        with torch.cuda.stream(s):
            buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _workspaces[key] = buf
    return buf


def release_workspaces(device=None, stream=None) -> int:
    """Drops the cached workspaces (all of them, or those of one device and/or
    stream) so torch can reuse their memory; returns how many were dropped.
    A server that makes a stream per request calls this when the stream is
    retired.  Work already queued keeps its buffer alive through torch's
    stream-ordered allocator."""
    torch = _torch()
    dev = None
    if device is not None:
        dev = torch.device(device)
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
    sid = None if stream is None else int(stream.cuda_stream)
    drop = [k for k in _workspaces if (dev is None or k[0] == str(dev)) and (sid is None or k[2] == sid)]
    for k in drop:
        del _workspaces[k]
    return len(drop)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_ptr(stream, device) -> int:
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}; the call runs on {device}")
    return stream.cuda_stream


def _on_device(device, **tensors) -> None:
    """Every tensor of one call lives on the GPU the call runs on (the library
    launches on the current device, which the entry points set to it)."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}; every tensor of the call must be on {device}")


def _ws(ws, nbytes: int, device, tag: str = "default", stream=None):
    """The caller's workspace (checked) or the stream's cached one, with its size in bytes."""
    torch = _torch()
    if ws is None:
        ws = workspace(nbytes, device, tag, stream)
    elif not isinstance(ws, torch.Tensor) or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {device}")
    return ws, ws.numel() * ws.element_size()


def _req(t, name, dtype, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device (no CPU path exists)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def prefill(q, k, v, q_gamma, k_gamma, positions, layer_kind: int, window: int, rope_base: float,
            interp_factor: float, image_spans=None, *, out=None, return_lse: bool = False,
            k_cache=None, v_cache=None, ws=None, stream=None):
    """One attention layer over full sequences; returns out (and lse).

    q [B,S,Hq,D] bf16, k/v [B,S,Hkv,D] bf16 (raw projections), gammas fp32
    [D], positions int32 [B,S], image_spans int32 [B,n,2] or None.
    """
    torch = _torch()
    _req(q, "q", torch.bfloat16)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    _req(k, "k", torch.bfloat16, (B, S, Hkv, D))
    _req(v, "v", torch.bfloat16, (B, S, Hkv, D))
    _req(q_gamma, "q_gamma", torch.float32, (D,))
    _req(k_gamma, "k_gamma", torch.float32, (D,))
    _req(positions, "positions", torch.int32, (B, S))
    n_spans = 0
    if image_spans is not None:
        _req(image_spans, "image_spans", torch.int32)
        if image_spans.dim() != 3 or image_spans.shape[0] != B or image_spans.shape[2] != 2:
            raise ValueError("image_spans must be [B, n, 2]")
        n_spans = int(image_spans.shape[1])
        if n_spans == 0:
            image_spans = None
    if out is None:
        out = torch.empty_like(q)
    _req(out, "out", torch.bfloat16, (B, S, Hq, D))
    lse = torch.empty(B, Hq, S, dtype=torch.float32, device=q.device) if return_lse else None
    cap = 0
    if k_cache is not None:
        _req(k_cache, "k_cache", torch.bfloat16)
        if k_cache.dim() != 4 or k_cache.shape[0] != B or k_cache.shape[1] != Hkv or k_cache.shape[3] != D:
            raise ValueError("k_cache must be [B, Hkv, capacity, D]")
        _req(v_cache, "v_cache", torch.bfloat16, tuple(k_cache.shape))
        cap = int(k_cache.shape[2])
    dev = q.device
    _on_device(dev, k=k, v=v, q_gamma=q_gamma, k_gamma=k_gamma, positions=positions, image_spans=image_spans,
               out=out, k_cache=k_cache, v_cache=v_cache)
    wsb, ws_bytes = _ws(ws, prefill_workspace_size(B, S, Hq, Hkv, D), dev, stream=stream)
    with torch.cuda.device(dev):
        st = lib().g3attn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(q_gamma), _ptr(k_gamma), _ptr(positions),
                                  int(layer_kind), int(window), float(rope_base), float(interp_factor),
                                  _ptr(image_spans), n_spans, B, S, Hq, Hkv, D, _ptr(out), _ptr(lse),
                                  _ptr(k_cache), _ptr(v_cache), cap, wsb.data_ptr(), ws_bytes,
                                  _stream_ptr(stream, dev))
    _check(st, "g3attn_prefill")
    return (out, lse) if return_lse else out


def prefill_backward(q, k, v, q_gamma, k_gamma, positions, layer_kind: int, window: int, rope_base: float,
                     interp_factor: float, image_spans, out, lse, dout, *, grads=None, ws=None, stream=None):
    """Gradients of one prefill layer: returns dict(dq, dk, dv, dq_gamma, dk_gamma).

    Arguments as for prefill, plus the forward's out [B,S,Hq,D] bf16 and lse
    [B,Hq,S] fp32 and the output gradient dout [B,S,Hq,D] bf16.  `grads` may
    hold preallocated outputs under the same keys.
    """
    torch = _torch()
    _req(q, "q", torch.bfloat16)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    _req(k, "k", torch.bfloat16, (B, S, Hkv, D))
    _req(v, "v", torch.bfloat16, (B, S, Hkv, D))
    _req(q_gamma, "q_gamma", torch.float32, (D,))
    _req(k_gamma, "k_gamma", torch.float32, (D,))
    _req(positions, "positions", torch.int32, (B, S))
    _req(out, "out", torch.bfloat16, (B, S, Hq, D))
    _req(lse, "lse", torch.float32, (B, Hq, S))
    _req(dout, "dout", torch.bfloat16, (B, S, Hq, D))
    n_spans = 0
    if image_spans is not None:
        _req(image_spans, "image_spans", torch.int32)
        if image_spans.dim() != 3 or image_spans.shape[0] != B or image_spans.shape[2] != 2:
            raise ValueError("image_spans must be [B, n, 2]")
        n_spans = int(image_spans.shape[1])
        if n_spans == 0:
            image_spans = None
    g = dict(grads) if grads is not None else {}
    g.setdefault("dq", torch.empty_like(q))
    g.setdefault("dk", torch.empty_like(k))
    g.setdefault("dv", torch.empty_like(v))
    g.setdefault("dq_gamma", torch.empty_like(q_gamma))
    g.setdefault("dk_gamma", torch.empty_like(k_gamma))
    _req(g["dq"], "dq", torch.bfloat16, (B, S, Hq, D))
    _req(g["dk"], "dk", torch.bfloat16, (B, S, Hkv, D))
    _req(g["dv"], "dv", torch.bfloat16, (B, S, Hkv, D))
    _req(g["dq_gamma"], "dq_gamma", torch.float32, (D,))
    _req(g["dk_gamma"], "dk_gamma", torch.float32, (D,))
    dev = q.device
    _on_device(dev, k=k, v=v, q_gamma=q_gamma, k_gamma=k_gamma, positions=positions, image_spans=image_spans,
               out=out, lse=lse, dout=dout, **g)
    wsb, ws_bytes = _ws(ws, prefill_backward_workspace_size(B, S, Hq, Hkv, D), dev, tag="backward",
                        stream=stream)
    with torch.cuda.device(dev):
        st = lib().g3attn_prefill_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(q_gamma), _ptr(k_gamma),
                                           _ptr(positions), int(layer_kind), int(window), float(rope_base),
                                           float(interp_factor), _ptr(image_spans), n_spans, B, S, Hq, Hkv, D,
                                           _ptr(out), _ptr(lse), _ptr(dout), _ptr(g["dq"]), _ptr(g["dk"]),
                                           _ptr(g["dv"]), _ptr(g["dq_gamma"]), _ptr(g["dk_gamma"]),
                                           wsb.data_ptr(), ws_bytes, _stream_ptr(stream, dev))
    _check(st, "g3attn_prefill_backward")
    return g


def decode(q, k_new, v_new, q_gamma, k_gamma, k_cache, v_cache, seq_lens, max_seq_len: int,
           layer_kind: int, window: int, rope_base: float, interp_factor: float, *, out=None,
           ws=None, stream=None):
    """One decode step: writes the new token into the cache and returns out [B,Hq,D]."""
    torch = _torch()
    _req(q, "q", torch.bfloat16)
    B, Hq, D = q.shape
    Hkv = k_new.shape[1]
    _req(k_new, "k_new", torch.bfloat16, (B, Hkv, D))
    _req(v_new, "v_new", torch.bfloat16, (B, Hkv, D))
    _req(q_gamma, "q_gamma", torch.float32, (D,))
    _req(k_gamma, "k_gamma", torch.float32, (D,))
    _req(k_cache, "k_cache", torch.bfloat16)
    cap = int(k_cache.shape[2])
    _req(k_cache, "k_cache", torch.bfloat16, (B, Hkv, cap, D))
    _req(v_cache, "v_cache", torch.bfloat16, (B, Hkv, cap, D))
    _req(seq_lens, "seq_lens", torch.int32, (B,))
    if out is None:
        out = torch.empty_like(q)
    _req(out, "out", torch.bfloat16, (B, Hq, D))
    dev = q.device
    _on_device(dev, k_new=k_new, v_new=v_new, q_gamma=q_gamma, k_gamma=k_gamma, k_cache=k_cache,
               v_cache=v_cache, seq_lens=seq_lens, out=out)
    # Decode keeps its own cached workspace: its launch clears the error word,
    # which would otherwise erase a prefill's unread device error.  A local
    # layer's query sees at most `window` ring slots, which bounds its scratch.
    visible = min(int(max_seq_len), int(window)) if layer_kind == LOCAL and window >= 1 else int(max_seq_len)
    wsb, ws_bytes = _ws(ws, decode_workspace_size(B, Hq, Hkv, D, visible), dev, tag="decode", stream=stream)
    with torch.cuda.device(dev):
        st = lib().g3attn_decode(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(q_gamma), _ptr(k_gamma),
                                 _ptr(k_cache), _ptr(v_cache), cap, _ptr(seq_lens), int(max_seq_len),
                                 int(layer_kind), int(window), float(rope_base), float(interp_factor),
                                 B, Hq, Hkv, D, _ptr(out), wsb.data_ptr(), ws_bytes, _stream_ptr(stream, dev))
    _check(st, "g3attn_decode")
    return out


def check_device_error(ws=None, device=None, stream=None) -> int:
    """Status recorded on the device by the last call using this workspace."""
    torch = _torch()
    if ws is None:
        dev = torch.device(device if device is not None else "cuda")
        ws = workspace(256, dev, stream=stream)
    if not isinstance(ws, torch.Tensor) or ws.device.type != "cuda":
        raise ValueError("ws must be a CUDA tensor")
    with torch.cuda.device(ws.device):
        return int(lib().g3attn_check_device_error(ws.data_ptr(), _stream_ptr(stream, ws.device)))


def trace_enable(on: bool = True) -> None:
    lib().g3attn_trace_enable(1 if on else 0)


def trace_collect() -> dict:
    arr = (KernelTrace * 32)()
    n = lib().g3attn_trace_collect(arr, 32)
    return {arr[i].name.decode(): (int(arr[i].launches), float(arr[i].total_ms)) for i in range(n)}


def prefill_chunk(q, k, v, q_gamma, k_gamma, positions, k_cache, v_cache, start: int, layer_kind: int,
                  window: int, rope_base: float, interp_factor: float, image_spans=None, *, out=None,
                  return_lse: bool = False, ws=None, stream=None):
    """The next C tokens of sequences whose first `start` tokens are cached; returns out (and lse).

    q [B,C,Hq,D] bf16, k/v [B,C,Hkv,D] bf16 (raw projections of the chunk),
    positions int32 [B,C], k_cache/v_cache bf16 [B,Hkv,cap,D] (updated in place),
    image_spans int32 [B,n,2] in whole-sequence token indices, or None.
    """
    torch = _torch()
    _req(q, "q", torch.bfloat16)
    B, C, Hq, D = q.shape
    Hkv = k.shape[2]
    _req(k, "k", torch.bfloat16, (B, C, Hkv, D))
    _req(v, "v", torch.bfloat16, (B, C, Hkv, D))
    _req(q_gamma, "q_gamma", torch.float32, (D,))
    _req(k_gamma, "k_gamma", torch.float32, (D,))
    _req(positions, "positions", torch.int32, (B, C))
    _req(k_cache, "k_cache", torch.bfloat16)
    _req(v_cache, "v_cache", torch.bfloat16, tuple(k_cache.shape))
    if k_cache.dim() != 4 or k_cache.shape[0] != B or k_cache.shape[1] != Hkv or k_cache.shape[3] != D:
        raise ValueError("k_cache must be [B, Hkv, capacity, D]")
    cap = int(k_cache.shape[2])
    n_spans = 0
    if image_spans is not None:
        _req(image_spans, "image_spans", torch.int32)
        if image_spans.dim() != 3 or image_spans.shape[0] != B or image_spans.shape[2] != 2:
            raise ValueError("image_spans must be [B, n, 2]")
        n_spans = int(image_spans.shape[1])
        if n_spans == 0:
            image_spans = None
    if out is None:
        out = torch.empty_like(q)
    _req(out, "out", torch.bfloat16, (B, C, Hq, D))
    lse = torch.empty(B, Hq, C, dtype=torch.float32, device=q.device) if return_lse else None
    need = prefill_chunk_workspace_size(B, C, Hq, Hkv, D, start, layer_kind, window)
    if need == 0:
        raise ValueError("invalid sizes for prefill_chunk")
    dev = q.device
    _on_device(dev, k=k, v=v, q_gamma=q_gamma, k_gamma=k_gamma, positions=positions, k_cache=k_cache,
               v_cache=v_cache, image_spans=image_spans, out=out)
    wsb, ws_bytes = _ws(ws, need, dev, stream=stream)
    with torch.cuda.device(dev):
        st = lib().g3attn_prefill_chunk(_ptr(q), _ptr(k), _ptr(v), _ptr(q_gamma), _ptr(k_gamma), _ptr(positions),
                                        _ptr(k_cache), _ptr(v_cache), cap, int(start), int(layer_kind),
                                        int(window), float(rope_base), float(interp_factor), _ptr(image_spans),
                                        n_spans, B, C, Hq, Hkv, D, _ptr(out), _ptr(lse), wsb.data_ptr(),
                                        ws_bytes, _stream_ptr(stream, dev))
    _check(st, "g3attn_prefill_chunk")
    return (out, lse) if return_lse else out


def soft_tokens(patches, gamma, grid_h: int, grid_w: int, pool: int = 4, *, out=None, stream=None):
    """Image soft tokens: pool x pool average of the patch grid, then RMS norm times gamma.

    patches bf16 [B, grid_h*grid_w, F], gamma fp32 [F]; returns bf16 [B, (grid_h/pool)*(grid_w/pool), F].
    """
    torch = _torch()
    _req(patches, "patches", torch.bfloat16)
    if patches.dim() != 3 or patches.shape[1] != grid_h * grid_w:
        raise ValueError("patches must be [B, grid_h * grid_w, F]")
    B, _, F = patches.shape
    _req(gamma, "gamma", torch.float32, (F,))
    n_out = (grid_h // pool) * (grid_w // pool)
    if out is None:
        out = torch.empty(B, n_out, F, dtype=torch.bfloat16, device=patches.device)
    _req(out, "out", torch.bfloat16, (B, n_out, F))
    dev = patches.device
    _on_device(dev, gamma=gamma, out=out)
    with torch.cuda.device(dev):
        st = lib().g3attn_soft_tokens(_ptr(patches), _ptr(gamma), B, grid_h, grid_w, F, pool, _ptr(out),
                                      _stream_ptr(stream, dev))
    _check(st, "g3attn_soft_tokens")
    return out


# ------------------------------------------------------------- paged cache
# A decode step makes several of these calls per layer, each a few microseconds
# on the GPU.  Where a call is plain (outputs made here, the current stream and
# device) the module _paged checks its arguments, allocates and calls the library;
# it answers None when something is not as expected, and the ordinary way below
# follows, which words the error or serves the options.
_paged_statuses = {}
_quick = None


class _Ordinary:
    """In the place of the module _paged where only the library was built: every call takes the ordinary way."""

    @staticmethod
    def _none(*args):
        return None

    page_map = paged_append = page_bounds = page_select = paged_decode = set_status = _none


def _load_quick():
    global _quick
    if _quick is None:
        lib()
        _torch()
        if os.path.exists(os.path.join(HERE, "_paged.so")):
            from . import _paged
            _quick = _paged
        else:
            _quick = _Ordinary  # first: where warnings are errors, the next call goes on
            warnings.warn("_paged.so is missing: each paged call takes 11 to 23 us of host time instead of 3 to 8 "
                          "(build it with `python -m global_gqa_b200.build`)", RuntimeWarning, stacklevel=3)
    return _quick


def paged_status(device=None):
    """The device's error words of the paged calls (int32 [2]), used where no `status` is given.

    Read and cleared by check_device_error(paged_status(device)).  Made on first
    use, which must be outside a stream capture.
    """
    torch = _torch()
    dev = torch.device("cuda" if device is None else device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    st = _paged_statuses.get(dev.index)
    if st is None:
        with torch.cuda.device(dev):
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("call paged_status() once before capturing paged calls, or give them a status")
            st = torch.zeros(2, dtype=torch.int32, device=dev)
            torch.cuda.current_stream(dev).synchronize()  # any stream may use it from now on
        st = _paged_statuses.setdefault(dev.index, st)
        _load_quick().set_status(dev.index, st)
    return st


def _arg(t, name, dtype, shape, device) -> int:
    """The address of a tensor argument; raises unless it is contiguous, of this type and shape, on this GPU."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _req(t, name, dtype, shape)
    _on_device(device, **{name: t})
    raise ValueError(f"{name} is not usable")


def _shape(t, name, n: int):
    """The shape of an argument that the others' shapes follow from (its type and place are left to _arg)."""
    try:
        shape = t.shape
    except AttributeError:
        raise TypeError(f"{name} must be a torch tensor") from None
    if len(shape) != n:
        raise ValueError(f"{name} must have {n} dimensions, got {tuple(shape)}")
    return shape


def _int32(v, name) -> int:
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:  # ctypes would drop the upper bits
        raise ValueError(f"{name}={v} does not fit in 32 bits")
    return v


def _gpu_of(t, name):
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device (no CPU path exists)")
    return dev


def _paged_call(fn, device, stream, status, *args) -> None:
    """One library call on `device`'s stream, with the status words and the stream appended."""
    torch = _torch()
    if status is None:
        status = _paged_statuses.get(device.index)
        if status is None:
            status = paged_status(device)
    st = _arg(status, "status", torch.int32, (2,), device)
    sp = _stream_ptr(stream, device)
    if torch.cuda.current_device() == device.index:
        code = getattr(_lib or lib(), fn)(*args, st, sp)
    else:
        with torch.cuda.device(device):
            code = getattr(_lib or lib(), fn)(*args, st, sp)
    if code != 0:
        _check(code, fn)


def _empty(stream, device, dtype, *shape):
    """An output or workspace whose memory belongs to the stream that the call runs on."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _stream_ptr(stream, device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def page_select_workspace_size(B: int, Hkv: int, max_pages: int) -> int:
    return int(lib().g3attn_page_select_workspace_size(B, Hkv, max_pages))


def paged_decode_workspace_size(D: int) -> int:
    return int(lib().g3attn_paged_decode_workspace_size(D))


def page_map(old_lens, new_lens, block_table, free_pages, free_state, page_size: int, n_pages: int, max_tokens: int, *,
             out=None, status=None, stream=None):
    """Block table entries (in place), slots and positions of one step's new tokens.

    old_lens, new_lens int32 [B] (tokens cached, tokens added), block_table int32
    [B, max_pages], free_pages int32 [capacity] (a ring of free page numbers),
    free_state int32 [2] (its head and count).  Returns dict(seq_lens [B],
    cu_tokens [B+1], slots [max_tokens], positions [max_tokens], free_state [2]),
    all int32; `out` may hold preallocated ones under the same keys.
    """
    if out is None and stream is None:
        r = (_quick or _load_quick()).page_map(old_lens, new_lens, block_table, free_pages, free_state, page_size, n_pages,
                                               max_tokens, status)
        if r is not None:
            return r
    i32 = _torch().int32
    _int32(max_tokens, "max_tokens")
    B, = _shape(old_lens, "old_lens", 1)
    max_pages = _shape(block_table, "block_table", 2)[1]
    cap, = _shape(free_pages, "free_pages", 1)
    dev = _gpu_of(old_lens, "old_lens")
    r = dict(out) if out is not None else {}
    for name, n in (("seq_lens", B), ("cu_tokens", B + 1), ("slots", max_tokens), ("positions", max_tokens),
                    ("free_state", 2)):
        if name not in r:
            r[name] = _empty(stream, dev, i32, n)
    _paged_call("g3attn_page_map", dev, stream, status, _arg(old_lens, "old_lens", i32, (B,), dev),
                _arg(new_lens, "new_lens", i32, (B,), dev), B,
                _arg(block_table, "block_table", i32, (B, max_pages), dev), max_pages,
                _arg(free_pages, "free_pages", i32, (cap,), dev), cap, _arg(free_state, "free_state", i32, (2,), dev),
                _int32(page_size, "page_size"), _int32(n_pages, "n_pages"), max_tokens,
                _arg(r["seq_lens"], "seq_lens", i32, (B,), dev),
                _arg(r["cu_tokens"], "cu_tokens", i32, (B + 1,), dev), _arg(r["slots"], "slots", i32, (max_tokens,), dev),
                _arg(r["positions"], "positions", i32, (max_tokens,), dev),
                _arg(r["free_state"], "out free_state", i32, (2,), dev))
    return r


def paged_append(k, v, k_gamma, positions, slots, k_pages, v_pages, rope_base: float, interp_factor: float, *, q=None,
                 q_gamma=None, q_hat=None, status=None, stream=None):
    """QK-norm and RoPE of T packed tokens: keys and values into their slots; returns q_hat (None without q).

    k, v bf16 [T,Hkv,D] and q bf16 [T,Hq,D] raw projections, gammas fp32 [D],
    positions and slots int32 [T] (slot below 0: not cached), k_pages/v_pages bf16
    [n_pages,Hkv,page_size,D] (updated in place).  Rows are packed as page_map's
    cu_tokens says, none for a sequence that waits: row b of what page_select and
    paged_decode take is
    q_hat.index_select(0, (cu_tokens[1:] - 1).clamp(min=0)), which is q_hat
    itself only where every sequence has one new token.
    """
    if q_hat is None and stream is None:
        r = (_quick or _load_quick()).paged_append(k, v, k_gamma, positions, slots, k_pages, v_pages, rope_base, interp_factor,
                                                   q, q_gamma, status)
        if r is not None:
            return None if r is True else r
    torch = _torch()
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    kv = T, Hkv, D = _shape(k, "k", 3)
    n_pages, _, P, _ = _shape(k_pages, "k_pages", 4)
    pool = (n_pages, Hkv, P, D)
    dev = _gpu_of(k, "k")
    Hq, pq, pg, ph = 0, None, None, None
    if q is not None:
        Hq = _shape(q, "q", 3)[1]
        pq, pg = _arg(q, "q", bf16, (T, Hq, D), dev), _arg(q_gamma, "q_gamma", f32, (D,), dev)
        if q_hat is None:
            q_hat = _empty(stream, dev, bf16, T, Hq, D)
        ph = _arg(q_hat, "q_hat", bf16, (T, Hq, D), dev)
    elif q_gamma is not None or q_hat is not None:
        raise ValueError("q_gamma and q_hat are given with q only")
    _paged_call("g3attn_paged_append", dev, stream, status, pq, _arg(k, "k", bf16, kv, dev), _arg(v, "v", bf16, kv, dev), pg,
                _arg(k_gamma, "k_gamma", f32, (D,), dev), _arg(positions, "positions", i32, (T,), dev),
                _arg(slots, "slots", i32, (T,), dev), _arg(k_pages, "k_pages", bf16, pool, dev),
                _arg(v_pages, "v_pages", bf16, pool, dev), n_pages, P, rope_base, interp_factor, T, Hq, Hkv, D, ph)
    return q_hat


def page_bounds(k_pages, block_table, old_lens, seq_lens, bounds, exps, *, status=None, stream=None):
    """Renews the key bounds of the pages that hold tokens old_lens .. seq_lens-1; returns (bounds, exps).

    k_pages bf16 [n_pages,Hkv,page_size,D], block_table int32 [B,max_pages],
    old_lens/seq_lens int32 [B]; bounds int8 [n_pages,Hkv,2,D] and exps int8
    [n_pages,Hkv], updated in place.
    """
    if stream is None and (_quick or _load_quick()).page_bounds(k_pages, block_table, old_lens, seq_lens, bounds, exps, status):
        return bounds, exps
    torch = _torch()
    i32, i8 = torch.int32, torch.int8
    pool = n_pages, Hkv, P, D = _shape(k_pages, "k_pages", 4)
    B, max_pages = _shape(block_table, "block_table", 2)
    dev = _gpu_of(k_pages, "k_pages")
    _paged_call("g3attn_page_bounds", dev, stream, status, _arg(k_pages, "k_pages", torch.bfloat16, pool, dev),
                _arg(block_table, "block_table", i32, (B, max_pages), dev), _arg(old_lens, "old_lens", i32, (B,), dev),
                _arg(seq_lens, "seq_lens", i32, (B,), dev), B, max_pages, n_pages, P, Hkv, D,
                _arg(bounds, "bounds", i8, (n_pages, Hkv, 2, D), dev), _arg(exps, "exps", i8, (n_pages, Hkv), dev))
    return bounds, exps


def page_select(q_hat, bounds, exps, block_table, seq_lens, page_size: int, n_select: int, *, out=None, ws=None,
                status=None, stream=None):
    """The newest page and the n_select-1 best-scored others of each (sequence, kv head), ascending, -1 behind.

    q_hat bf16 [B,Hq,D], row b for sequence b (see paged_append), bounds/exps from
    page_bounds; returns
    int32 [B,Hkv,n_select], for paged_decode(pages=...).
    """
    if out is None and ws is None and stream is None:
        r = (_quick or _load_quick()).page_select(q_hat, bounds, exps, block_table, seq_lens, page_size, n_select, status)
        if r is not None:
            return r
    torch = _torch()
    i32, i8 = torch.int32, torch.int8
    B, Hq, D = _shape(q_hat, "q_hat", 3)
    n_pages, Hkv = _shape(exps, "exps", 2)
    max_pages = _shape(block_table, "block_table", 2)[1]
    dev = _gpu_of(q_hat, "q_hat")
    if out is None:
        out = _empty(stream, dev, i32, B, Hkv, max(_int32(n_select, "n_select"), 0))
    if ws is None:
        ws = _empty(stream, dev, torch.uint8, max(page_select_workspace_size(B, Hkv, max_pages), 1))
    ws, ws_bytes = _ws(ws, 0, dev)
    _paged_call("g3attn_page_select", dev, stream, status, _arg(q_hat, "q_hat", torch.bfloat16, (B, Hq, D), dev),
                _arg(bounds, "bounds", i8, (n_pages, Hkv, 2, D), dev), _arg(exps, "exps", i8, (n_pages, Hkv), dev),
                _arg(block_table, "block_table", i32, (B, max_pages), dev), _arg(seq_lens, "seq_lens", i32, (B,), dev), B,
                max_pages, n_pages, _int32(page_size, "page_size"), Hq, Hkv, D, n_select, _arg(out, "out", i32, (B, Hkv, n_select), dev),
                ws.data_ptr(), ws_bytes)
    return out


def paged_decode(q_hat, k_pages, v_pages, block_table, seq_lens, layer_kind: int, window: int, *, pages=None, out=None,
                 return_lse: bool = False, ws=None, status=None, stream=None):
    """Attention of one new token per sequence over its pages; returns out [B,Hq,D] (and lse [B,Hq]).

    q_hat bf16 [B,Hq,D], row b for sequence b (see paged_append), k_pages/v_pages
    bf16 [n_pages,Hkv,page_size,D], block_table int32 [B,max_pages], seq_lens int32 [B]
    (the new token included; 0: idle, a zero row), pages int32 [B,Hkv,n] from
    page_select or None (all pages; the last `window` tokens on a LOCAL layer).
    """
    if out is None and ws is None and stream is None:
        r = (_quick or _load_quick()).paged_decode(q_hat, k_pages, v_pages, block_table, seq_lens, layer_kind, window, pages,
                                                   return_lse, status)
        if r is not None:
            return r
    torch = _torch()
    bf16, i32 = torch.bfloat16, torch.int32
    B, Hq, D = _shape(q_hat, "q_hat", 3)
    dev = _gpu_of(q_hat, "q_hat")
    n_pages, Hkv, P, _ = _shape(k_pages, "k_pages", 4)
    max_pages = _shape(block_table, "block_table", 2)[1]
    pool = (n_pages, Hkv, P, D)
    n_select, plist = 0, None
    if pages is not None:
        n_select = _shape(pages, "pages", 3)[2]
        if n_select == 0:
            raise ValueError("pages has no entries (None attends to all pages)")
        plist = _arg(pages, "pages", i32, (B, Hkv, n_select), dev)
    if out is None:
        out = _empty(stream, dev, bf16, B, Hq, D)
    lse = _empty(stream, dev, torch.float32, B, Hq) if return_lse else None
    if ws is None:
        ws = _empty(stream, dev, torch.uint8, max(paged_decode_workspace_size(D), 1))
    ws, ws_bytes = _ws(ws, 0, dev)
    _paged_call("g3attn_paged_decode", dev, stream, status, _arg(q_hat, "q_hat", bf16, (B, Hq, D), dev),
                _arg(k_pages, "k_pages", bf16, pool, dev), _arg(v_pages, "v_pages", bf16, pool, dev),
                _arg(block_table, "block_table", i32, (B, max_pages), dev), _arg(seq_lens, "seq_lens", i32, (B,), dev), plist,
                n_select, _int32(layer_kind, "layer_kind"), _int32(window, "window"), B, max_pages, n_pages, P, Hq, Hkv, D,
                _arg(out, "out", bf16, (B, Hq, D), dev), _ptr(lse), ws.data_ptr(), ws_bytes)
    return (out, lse) if return_lse else out
