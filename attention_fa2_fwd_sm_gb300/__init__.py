"""Python binding of libattn.so (fused attention for GB300 / sm_103a).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/attn.h``.  The functions take
torch tensors (for device memory and the current stream) and return the
library's status code; ``check`` turns a non-zero code into an exception.
There is no fallback: if ``libattn.so`` cannot be loaded, importing the
functions raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libattn.so")

ATTN_OK = 0
ATTN_ERR_ARG = -1
ATTN_ERR_UNSUPPORTED = -2
ATTN_ERR_WORKSPACE = -3
ATTN_ERR_CUDA = -4
ATTN_ERR_TIMEOUT = -5

ORDER_HEAD_FIRST = 0
ORDER_BLOCK_FIRST = 1
ORDER_NAIVE_HEAD_FIRST = 2
ORDER_DIE_SPLIT_HEAD_FIRST = 3
ORDERS = {"head_first": ORDER_HEAD_FIRST, "block_first": ORDER_BLOCK_FIRST,
          "naive_head_first": ORDER_NAIVE_HEAD_FIRST,
          "die_split_head_first": ORDER_DIE_SPLIT_HEAD_FIRST}
# forward tile schemes, OR-ed into tile_order (0: the library's choice)
FWD_SINGLE_CTA = 0x100
FWD_CTA_PAIR = 0x200
# frequency rules of rope_freqs
ROPE_RULES = {"plain": 0, "linear": 1, "base": 2, "by_parts": 3}
SCHEMES = {"auto": 0, "single": FWD_SINGLE_CTA, "pair": FWD_CTA_PAIR}

# Every symbol include/attn.h declares, with (restype, argtypes).
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_LL = ctypes.c_longlong
_SZ = ctypes.c_size_t
_IP = ctypes.POINTER(ctypes.c_int)
_FP = ctypes.POINTER(ctypes.c_float)
_D = ctypes.c_double
_DP = ctypes.POINTER(ctypes.c_double)
SIGNATURES = {
    "attn_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P]),
    "attn_fwd_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _I, _P]),
    "attn_fwd_host": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _I, _I, _P, _SZ, _P]),
    "attn_fwd_host_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "attn_fwd_splitkv": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _I, _P, _SZ, _P]),
    "attn_fwd_splitkv_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "attn_fwd_host_trace": (_I, [_I]),
    "attn_fwd_host_trace_read": (_LL, [_FP, _LL]),
    "attn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _I, _P, _SZ, _P]),
    "attn_bwd_workspace_bytes": (_SZ, [_I, _I, _I]),
    "attn_bwd_workspace_bytes_ex": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "attn_decode": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _I, _P, _SZ, _P]),
    "attn_decode_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _I, _P]),
    "attn_decode_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "attn_decode_varlen": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _SZ, _P]),
    "attn_decode_varlen_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "attn_decode_num_splits": (_I, [_I, _I, _I, _I]),
    "attn_rope": (_I, [_P, _P, _P, _P, _P, _LL, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _P]),
    "attn_rope_freqs": (_I, [_DP, _I, _D, _I, _D, _D, _D, _D]),
    "attn_rope_append": (_I, [_P] * 13 + [_I] * 7 + [_F, _I, _P, _P]),
    "attn_decode_prefix": (_I, [_P] * 9 + [_I] * 5 + [_F, _I, _P, _SZ, _P]),
    "attn_decode_prefix_workspace_bytes": (_SZ, [_I] * 7),
    "attn_decode_prefix_segment": (_I, [_I] * 6 + [_LL] + [_I] * 3 + [_IP]),
    "attn_cache_evict": (_I, [_P] * 11 + [_I] * 7 + [_P, _SZ, _P]),
    "attn_cache_evict_workspace_bytes": (_SZ, [_I] * 5),
    "attn_tile_map": (_I, [_I, _I, _I, _I, _I, _I, _LL, _IP, _IP, _IP]),
    "attn_tile_map_die_split": (_I, [_I, _I, _I, _I, _I, _I, _LL, _IP, _IP, _IP]),
    "attn_bwd_tile_map": (_I, [_I, _I, _I, _I, _I, _I, _LL, _IP, _IP, _IP]),
    "attn_die_map": (_I, [_IP, _I, _FP]),
    "attn_fwd_units": (_LL, [_I, _I, _I]),
    "attn_device_status": (_I, [_P]),
    "attn_set_wait_timeout_ns": (_LL, [_LL]),
    "attn_strerror": (ctypes.c_char_p, [_I]),
    "attn_last_error": (ctypes.c_char_p, []),
    "attn_version": (_I, []),
}

_lib = None


class AttnError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        msg = f"{what}: {strerror(code)} ({code})" if what else f"{strerror(code)} ({code})"
        if code == ATTN_ERR_CUDA:
            msg += f" [{attn_last_error()}]"
        super().__init__(msg)


def lib():
    """Load libattn.so (raises OSError / RuntimeError when it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "attention_fa2_fwd_sm_gb300._build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().attn_strerror(int(code)).decode()


def check(code: int, what: str = "") -> None:
    if code != ATTN_OK:
        raise AttnError(code, what)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def attn_fwd(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, causal, stream=None) -> int:
    return lib().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d,
                          float(scale), int(bool(causal)), _stream(stream))


def attn_fwd_ex(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, causal, tile_order, stream=None) -> int:
    return lib().attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d,
                             float(scale), int(bool(causal)), int(tile_order), _stream(stream))


def attn_fwd_host(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, causal, tile_order, kv_heads_per_chunk,
                  workspace, workspace_bytes, stream=None) -> int:
    return lib().attn_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d, float(scale),
                               int(bool(causal)), int(tile_order), int(kv_heads_per_chunk), _ptr(workspace),
                               int(workspace_bytes), _stream(stream))


def attn_fwd_host_workspace_bytes(B, Hq, Hkv, N, d, kv_heads_per_chunk=0) -> int:
    return int(lib().attn_fwd_host_workspace_bytes(B, Hq, Hkv, N, d, kv_heads_per_chunk))


def attn_fwd_splitkv(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, causal, kv_splits, workspace, workspace_bytes,
                     stream=None) -> int:
    return lib().attn_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d, float(scale),
                                  int(bool(causal)), int(kv_splits), _ptr(workspace), int(workspace_bytes),
                                  _stream(stream))


def attn_fwd_splitkv_workspace_bytes(B, Hq, N, d, kv_splits=0) -> int:
    return int(lib().attn_fwd_splitkv_workspace_bytes(B, Hq, N, d, kv_splits))


def forward_splitkv(q, k, v, causal=False, scale=None, kv_splits=0, workspace=None, with_lse=True, stream=None):
    """Allocate outputs (and a workspace when none is given) and run
    attn_fwd_splitkv on ``[B, H, N, d]`` bf16 CUDA tensors; returns
    ``(o, lse, workspace)``."""
    import torch
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    if scale is None:
        scale = d ** -0.5
    nbytes = attn_fwd_splitkv_workspace_bytes(B, Hq, N, d, kv_splits)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if with_lse else None
    check(attn_fwd_splitkv(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, causal, kv_splits, workspace, nbytes,
                           stream), "attn_fwd_splitkv")
    return o, lse, workspace


def attn_fwd_host_trace(enable) -> int:
    return int(lib().attn_fwd_host_trace(int(bool(enable))))


def attn_fwd_host_trace_read(capacity=None):
    """Per-chunk timeline of the last traced attn_fwd_host call on the current
    device: a list of (copy-in done, kernel reached, kernel done, copy-out
    done) in ms from the call's start.  Raises when there is none."""
    n = int(lib().attn_fwd_host_trace_read(None, 0))
    if n < 0:
        check(n, "attn_fwd_host_trace_read")
    cap = n if capacity is None else min(n, int(capacity))
    buf = (ctypes.c_float * (4 * max(cap, 1)))()
    got = int(lib().attn_fwd_host_trace_read(buf, cap))
    if got < 0:
        check(got, "attn_fwd_host_trace_read")
    return [tuple(buf[4 * c: 4 * c + 4]) for c in range(cap)]


def attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, causal, tile_order,
             workspace, workspace_bytes, stream=None) -> int:
    return lib().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                          _ptr(dv), B, Hq, Hkv, N, d, float(scale), int(bool(causal)), int(tile_order),
                          _ptr(workspace), int(workspace_bytes), _stream(stream))


def attn_bwd_workspace_bytes(B, Hq, N) -> int:
    return int(lib().attn_bwd_workspace_bytes(B, Hq, N))


def attn_bwd_workspace_bytes_ex(B, Hq, Hkv, N, d, causal) -> int:
    return int(lib().attn_bwd_workspace_bytes_ex(B, Hq, Hkv, N, d, int(bool(causal))))


def attn_decode(q, kcache, vcache, seqlens, o, B, Hq, Hkv, d, scale, num_splits, max_seqlen,
                workspace=None, workspace_bytes=0, stream=None) -> int:
    return lib().attn_decode(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(seqlens), _ptr(o), B, Hq,
                             Hkv, d, float(scale), int(num_splits), int(max_seqlen),
                             _ptr(workspace), int(workspace_bytes), _stream(stream))


def attn_decode_noalloc(q, kcache, vcache, seqlens, o, B, Hq, Hkv, d, scale, num_splits, max_seqlen,
                        stream=None) -> int:
    """attn_decode for callers that cannot allocate device memory: the split
    partials go to a scratch array built into the library (see attn.h)."""
    return lib().attn_decode_noalloc(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(seqlens), _ptr(o), B,
                                     Hq, Hkv, d, float(scale), int(num_splits), int(max_seqlen),
                                     _stream(stream))


DECODE_NOALLOC_SCRATCH_BYTES = 4194304


def attn_decode_varlen(q, kcache, vcache, seqlens, o, B, Hq, Hkv, d, scale, max_seqlen, workspace,
                       workspace_bytes, stream=None) -> int:
    return lib().attn_decode_varlen(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(seqlens), _ptr(o), B, Hq, Hkv,
                                    d, float(scale), int(max_seqlen), _ptr(workspace), int(workspace_bytes),
                                    _stream(stream))


def attn_decode_varlen_workspace_bytes(B, Hq, Hkv, d) -> int:
    return int(lib().attn_decode_varlen_workspace_bytes(B, Hq, Hkv, d))


def decode_varlen(q, kcache, vcache, seqlens, scale=None, workspace=None, stream=None):
    """Allocate the output (and a workspace when none is given) and run
    attn_decode_varlen; returns ``(o, workspace)``."""
    import torch
    B, Hq, d = q.shape
    Hkv, s_max = kcache.shape[1], kcache.shape[2]
    if scale is None:
        scale = d ** -0.5
    nbytes = attn_decode_varlen_workspace_bytes(B, Hq, Hkv, d)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    check(attn_decode_varlen(q, kcache, vcache, seqlens, o, B, Hq, Hkv, d, scale, s_max, workspace,
                             workspace.numel(), stream), "attn_decode_varlen")
    return o, workspace


def attn_decode_workspace_bytes(B, Hq, d, num_splits) -> int:
    return int(lib().attn_decode_workspace_bytes(B, Hq, d, num_splits))


def attn_decode_num_splits(B, Hq, Hkv, max_seqlen) -> int:
    return int(lib().attn_decode_num_splits(B, Hq, Hkv, max_seqlen))


def attn_tile_map(tile_order, B, Hq, Hkv, N, causal, unit):
    b, h, m = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    rc = lib().attn_tile_map(int(tile_order), B, Hq, Hkv, N, int(bool(causal)), int(unit),
                             ctypes.byref(b), ctypes.byref(h), ctypes.byref(m))
    check(rc, "attn_tile_map")
    return b.value, h.value, m.value


def attn_tile_map_die_split(B, Hq, Hkv, N, causal, die, k):
    """(b, h, m) of the k-th unit of die `die` under the die-split order, or
    None when that die has no k-th unit of its own."""
    b, h, m = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    rc = lib().attn_tile_map_die_split(B, Hq, Hkv, N, int(bool(causal)), int(die), int(k),
                                       ctypes.byref(b), ctypes.byref(h), ctypes.byref(m))
    if rc == ATTN_ERR_ARG:
        return None
    check(rc, "attn_tile_map_die_split")
    return b.value, h.value, m.value


def attn_bwd_tile_map(tile_order, B, Hkv, N, causal, num_sms, unit):
    """(b, g, j) of dK/dV unit `unit`: batch entry, KV head, 128-key block."""
    b, g, j = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    rc = lib().attn_bwd_tile_map(int(tile_order), B, Hkv, N, int(bool(causal)), int(num_sms), int(unit),
                                 ctypes.byref(b), ctypes.byref(g), ctypes.byref(j))
    check(rc, "attn_bwd_tile_map")
    return b.value, g.value, j.value


def attn_die_map(capacity=256):
    """(die of each SM id, stats) of the current device, as the die-split order
    uses it; stats = (measured, min |corr|, near clk, far clk)."""
    dies = (ctypes.c_int * capacity)()
    stats = (ctypes.c_float * 4)()
    n = lib().attn_die_map(dies, capacity, stats)
    if n < 0:
        check(n, "attn_die_map")
    return list(dies[:min(n, capacity)]), tuple(stats)


def attn_fwd_units(B, Hq, N) -> int:
    return int(lib().attn_fwd_units(B, Hq, N))


def attn_device_status(stream=None) -> int:
    return lib().attn_device_status(_stream(stream))


def attn_set_wait_timeout_ns(ns: int) -> int:
    return int(lib().attn_set_wait_timeout_ns(int(ns)))


def attn_last_error() -> str:
    return lib().attn_last_error().decode()


def attn_version() -> int:
    return int(lib().attn_version())


_strides = struct.Struct("12q").pack  # a host array: (batch, head, token) element strides of four tensors


def attn_rope(q, q_out, k, k_out, positions, position_stride, inv_freq, B, Hq, Hkv, N, d, rotary_dim, interleaved,
              out_scale, inverse, strides=None, stream=None) -> int:
    return lib().attn_rope(_ptr(q), _ptr(q_out), _ptr(k), _ptr(k_out), _ptr(positions), position_stride,
                           _ptr(inv_freq), B, Hq, Hkv, N, d, rotary_dim, int(bool(interleaved)), out_scale,
                           int(bool(inverse)), strides, _stream(stream))


def attn_rope_append(q, q_out, k, v, kcache, vcache, seqlens, start_pos, new_lens, seqlens_out, cache_pos, weights,
                     inv_freq, B, Hq, Hkv, T, d, rotary_dim, interleaved, out_scale, max_seqlen, strides=None,
                     stream=None) -> int:
    return lib().attn_rope_append(_ptr(q), _ptr(q_out), _ptr(k), _ptr(v), _ptr(kcache), _ptr(vcache), _ptr(seqlens),
                                  _ptr(start_pos), _ptr(new_lens), _ptr(seqlens_out), _ptr(cache_pos), _ptr(weights),
                                  _ptr(inv_freq), B, Hq, Hkv, T, d, rotary_dim, int(bool(interleaved)), out_scale,
                                  max_seqlen, strides, _stream(stream))


def attn_decode_prefix(q, kprefix, vprefix, kcache, vcache, seqlens, o, lse, weights, B, Hq, Hkv, P, d, scale,
                       max_seqlen, workspace, workspace_bytes, stream=None) -> int:
    return lib().attn_decode_prefix(_ptr(q), _ptr(kprefix), _ptr(vprefix), _ptr(kcache), _ptr(vcache), _ptr(seqlens),
                                    _ptr(o), _ptr(lse), _ptr(weights), B, Hq, Hkv, P, d, scale, max_seqlen,
                                    _ptr(workspace), workspace_bytes, _stream(stream))


def attn_decode_prefix_workspace_bytes(B, Hq, Hkv, P, d, max_seqlen, with_weights=False) -> int:
    return lib().attn_decode_prefix_workspace_bytes(B, Hq, Hkv, P, d, max_seqlen, int(bool(with_weights)))


def attn_decode_prefix_segment(B, Hq, Hkv, P, d, max_seqlen, own_keys, num_sms, cta, i):
    """(KV head, unit, first key block, blocks, partial, its rows' last partial)
    of CTA `cta`'s i-th piece of the prefix phase, or None when it has no i-th
    piece."""
    out = (ctypes.c_int * 6)()
    rc = lib().attn_decode_prefix_segment(B, Hq, Hkv, P, d, max_seqlen, own_keys, num_sms, cta, i, out)
    if rc < 0:
        check(rc, "attn_decode_prefix_segment")
    return tuple(out) if rc else None


def attn_cache_evict(kcache, vcache, weights, cache_pos, seqlens, cur_pos, kout, vout, weights_out, pos_out,
                     seqlens_out, B, Hkv, d, max_seqlen, out_seqlen, keep, recent, workspace, workspace_bytes,
                     stream=None) -> int:
    return lib().attn_cache_evict(_ptr(kcache), _ptr(vcache), _ptr(weights), _ptr(cache_pos), _ptr(seqlens),
                                  _ptr(cur_pos), _ptr(kout), _ptr(vout), _ptr(weights_out), _ptr(pos_out),
                                  _ptr(seqlens_out), B, Hkv, d, max_seqlen, out_seqlen, keep, recent, _ptr(workspace),
                                  workspace_bytes, _stream(stream))


def attn_cache_evict_workspace_bytes(B, Hkv, max_seqlen, keep, in_place) -> int:
    return lib().attn_cache_evict_workspace_bytes(B, Hkv, max_seqlen, keep, int(bool(in_place)))


def attn_rope_freqs(rotary_dim, base=10000.0, rule=0, factor=1.0, low=1.0, high=4.0, trained_len=8192.0):
    """List of rotary_dim / 2 frequencies (radians per position) by one of ROPE_RULES."""
    buf = (ctypes.c_double * max(int(rotary_dim) // 2, 1))()
    check(lib().attn_rope_freqs(buf, int(rotary_dim), base, int(rule), factor, low, high, trained_len),
          "attn_rope_freqs")
    return list(buf)


# ----------------------------------------------------------- torch helpers
def _fits(t, dtype, shape, gpu):
    """A contiguous tensor of this type and shape on this GPU."""
    return t is not None and t.dtype is dtype and t.shape == shape and t.get_device() == gpu and t.is_contiguous()


def _fits_rows(t, dtype, shape, gpu):
    """The same with any strides, columns contiguous."""
    return t is not None and t.dtype is dtype and t.shape == shape and t.get_device() == gpu and t.stride(-1) == 1


def _refuse(what, name, t, dtype, shape):
    """ATTN_ERR_ARG for a tensor that the call cannot take as it is: its
    address alone would not tell the library."""
    got = "None" if t is None else f"{t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}"
    raise AttnError(ATTN_ERR_ARG, f"{what}: {name} has to be {dtype} {tuple(shape)}, on the GPU of the first tensor, with "
                                  f"contiguous rows (got {got})")


def _elsewhere(what, gpu, stream):
    """The context that makes `stream` (or GPU `gpu`'s current one) the current
    stream.  The helpers below call themselves inside it unless it is current
    already, so the outputs and workspaces that they allocate belong to the
    stream that writes them."""
    import torch
    if gpu < 0:
        raise AttnError(ATTN_ERR_ARG, f"{what}: the tensors have to be on a GPU")
    if stream is None:
        return torch.cuda.device(gpu)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=gpu) if stream else torch.cuda.default_stream(gpu)
    if stream.device.index != gpu:
        raise AttnError(ATTN_ERR_ARG, f"{what}: the stream belongs to {stream.device}, the tensors to cuda:{gpu}")
    return torch.cuda.stream(stream)


def _lend(stream, *tensors):
    """Tell the allocator that `stream` uses these tensors, so that none of them is
    given away under its kernels when the caller lets go of it.  Not for a
    stream that torch does not own: it may be gone by then."""
    import torch
    if isinstance(stream, torch.cuda.Stream) and not isinstance(stream, torch.cuda.ExternalStream):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _held(what, workspace, gpu):
    """Bytes of the caller's workspace."""
    if workspace.get_device() != gpu or not workspace.is_contiguous():
        raise AttnError(ATTN_ERR_WORKSPACE, f"{what}: the workspace has to be contiguous and on the tensors' GPU")
    return workspace.nbytes


def rope_freqs(rotary_dim, base=10000.0, rule="plain", factor=1.0, low=1.0, high=4.0, trained_len=8192.0,
               device=None):
    """The frequencies of attn_rope_freqs as an fp64 CUDA tensor, for `rope`
    and `rope_append` (make it once and keep it)."""
    import torch
    f = attn_rope_freqs(rotary_dim, base, ROPE_RULES[rule], factor, low, high, trained_len)
    return torch.tensor(f, dtype=torch.float64, device="cuda" if device is None else device)


def rope(q, k, inv_freq, positions=None, interleaved=False, out_scale=1.0, out=None, inverse=False, stream=None):
    """Rotate ``[B, H, N, d]`` bf16 CUDA tensors (any strides with contiguous
    columns, so a fused projection's views too) by attn_rope; `k` may be None.
    `positions` is ``[N]`` or ``[B, N]`` int32, or None for 0..N-1; rotary_dim
    is twice the length of `inv_freq`.  Returns ``(q_out, k_out)``: contiguous
    tensors as attn_fwd takes them, or `out`, which may be ``(q, k)``.

    `stream` (here and in the other decode-cache helpers): a torch stream, or
    an address of one, other than the current one.  What the call allocates
    belongs to it.  The inputs are kept for it by the allocator where the stream
    is torch's own; the caller keeps them until the work is done where it is an
    address or a torch.cuda.ExternalStream."""
    import torch
    what, bf16 = "rope", torch.bfloat16
    gpu = q.get_device()
    if stream is not None or gpu < 0 or gpu != torch._C._cuda_getDevice():
        with _elsewhere(what, gpu, stream):
            got = rope(q, k, inv_freq, positions, interleaved, out_scale, out, inverse)
        _lend(stream, q, k, inv_freq, positions, *(out or ()))
        return got
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise AttnError(ATTN_ERR_ARG, "rope: q and k have to be [B, H, N, d]")
    B, Hq, N, d = q.shape
    pairs = inv_freq.numel()
    _fits_rows(q, bf16, q.shape, gpu) or _refuse(what, "q", q, bf16, q.shape)
    _fits(inv_freq, torch.float64, (pairs,), gpu) or _refuse(what, "inv_freq", inv_freq, torch.float64, (pairs,))
    per_entry = 0
    if positions is not None:
        shape = (N,)
        if positions.dim() == 2:
            per_entry, shape = N, (B, N)
        _fits(positions, torch.int32, shape, gpu) or _refuse(what, "positions", positions, torch.int32, shape)
    q_out, k_out = (None, None) if out is None else out
    if out is not None and (q_out is None or (k is None) != (k_out is None)):
        raise AttnError(ATTN_ERR_ARG, "rope: out has to hold q_out, and k_out exactly where there is a k")
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _fits_rows(q_out, bf16, q.shape, gpu) or _refuse(what, "q_out", q_out, bf16, q.shape)
    Hkv, ks, kos = 0, (0, 0, 0, 1), (0, 0, 0, 1)
    if k is not None:
        Hkv = k.shape[1]
        shape = (B, Hkv, N, d)
        _fits_rows(k, bf16, shape, gpu) or _refuse(what, "k", k, bf16, shape)
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        else:
            _fits_rows(k_out, bf16, shape, gpu) or _refuse(what, "k_out", k_out, bf16, shape)
        ks, kos = k.stride(), k_out.stride()
    rc = lib().attn_rope(q.data_ptr(), q_out.data_ptr(), None if k is None else k.data_ptr(),
                         None if k is None else k_out.data_ptr(), None if positions is None else positions.data_ptr(),
                         per_entry, inv_freq.data_ptr(), B, Hq, Hkv, N, d, 2 * pairs, interleaved, out_scale, inverse,
                         _strides(*q.stride()[:3], *q_out.stride()[:3], *ks[:3], *kos[:3]),
                         torch._C._cuda_getCurrentRawStream(gpu))
    if rc:
        check(rc, "attn_rope")
    return q_out, k_out


def rope_backward(dq, dk, inv_freq, positions=None, interleaved=False, out_scale=1.0, out=None, stream=None):
    """Gradients of `rope` (the arguments it was called with): from those of
    its outputs to those of its inputs; returns ``(dq_in, dk_in)``."""
    return rope(dq, dk, inv_freq, positions, interleaved, out_scale, out, True, stream)


def rope_append(q, k, v, kcache, vcache, seqlens, inv_freq=None, start_pos=None, new_lens=None, interleaved=False,
                out_scale=1.0, cache_pos=None, weights=None, q_out=None, seqlens_out=None, stream=None):
    """Rotate the new tokens' q ``[B, Hq, T, d]`` and append their rotated k
    and their v ``[B, Hkv, T, d]`` (any strides with contiguous columns) to the
    caches by attn_rope_append; without `inv_freq` nothing is rotated.
    Allocates the outputs that are not given; returns ``(q_out,
    seqlens_out)``."""
    import torch
    what, bf16, i32 = "rope_append", torch.bfloat16, torch.int32
    gpu = q.get_device()
    if stream is not None or gpu < 0 or gpu != torch._C._cuda_getDevice():
        with _elsewhere(what, gpu, stream):
            got = rope_append(q, k, v, kcache, vcache, seqlens, inv_freq, start_pos, new_lens, interleaved, out_scale,
                              cache_pos, weights, q_out, seqlens_out)
        _lend(stream, q, k, v, kcache, vcache, seqlens, inv_freq, start_pos, new_lens, cache_pos, weights, q_out,
              seqlens_out)
        return got
    if q.dim() != 4 or kcache.dim() != 4:
        raise AttnError(ATTN_ERR_ARG, "rope_append: q has to be [B, Hq, T, d], the caches [B, Hkv, max_seqlen, d]")
    B, Hq, T, d = q.shape
    Hkv, s_max = kcache.shape[1], kcache.shape[2]
    new, cache, per_key = (B, Hkv, T, d), (B, Hkv, s_max, d), (B, Hkv, s_max)
    _fits_rows(q, bf16, q.shape, gpu) or _refuse(what, "q", q, bf16, q.shape)
    _fits_rows(k, bf16, new, gpu) or _refuse(what, "k", k, bf16, new)
    _fits_rows(v, bf16, new, gpu) or _refuse(what, "v", v, bf16, new)
    _fits(kcache, bf16, cache, gpu) or _refuse(what, "kcache", kcache, bf16, cache)
    _fits(vcache, bf16, cache, gpu) or _refuse(what, "vcache", vcache, bf16, cache)
    _fits(seqlens, i32, (B,), gpu) or _refuse(what, "seqlens", seqlens, i32, (B,))
    start_pos is None or _fits(start_pos, i32, (B,), gpu) or _refuse(what, "start_pos", start_pos, i32, (B,))
    new_lens is None or _fits(new_lens, i32, (B,), gpu) or _refuse(what, "new_lens", new_lens, i32, (B,))
    cache_pos is None or _fits(cache_pos, i32, per_key, gpu) or _refuse(what, "cache_pos", cache_pos, i32, per_key)
    weights is None or _fits(weights, torch.float32, per_key, gpu) or _refuse(what, "weights", weights, torch.float32,
                                                                              per_key)
    rotary_dim = 0
    if inv_freq is not None:
        pairs = inv_freq.numel()
        rotary_dim = 2 * pairs
        _fits(inv_freq, torch.float64, (pairs,), gpu) or _refuse(what, "inv_freq", inv_freq, torch.float64, (pairs,))
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _fits_rows(q_out, bf16, q.shape, gpu) or _refuse(what, "q_out", q_out, bf16, q.shape)
    if seqlens_out is None:
        seqlens_out = torch.empty_like(seqlens)
    else:
        _fits(seqlens_out, i32, (B,), gpu) or _refuse(what, "seqlens_out", seqlens_out, i32, (B,))
    rc = lib().attn_rope_append(q.data_ptr(), q_out.data_ptr(), k.data_ptr(), v.data_ptr(), kcache.data_ptr(),
                                vcache.data_ptr(), seqlens.data_ptr(), None if start_pos is None else start_pos.data_ptr(),
                                None if new_lens is None else new_lens.data_ptr(), seqlens_out.data_ptr(),
                                None if cache_pos is None else cache_pos.data_ptr(),
                                None if weights is None else weights.data_ptr(),
                                None if inv_freq is None else inv_freq.data_ptr(), B, Hq, Hkv, T, d, rotary_dim,
                                interleaved, out_scale, s_max,
                                _strides(*q.stride()[:3], *q_out.stride()[:3], *k.stride()[:3], *v.stride()[:3]),
                                torch._C._cuda_getCurrentRawStream(gpu))
    if rc:
        check(rc, "attn_rope_append")
    return q_out, seqlens_out


def decode_prefix(q, kprefix, vprefix, kcache, vcache, seqlens, scale=None, weights=None, workspace=None,
                  with_lse=True, stream=None):
    """One decode step by attn_decode_prefix: q ``[B, Hq, d]`` over a prefix
    ``[Hkv, P, d]`` that the batch shares (None: none) and the sequences' own
    caches ``[B, Hkv, max_seqlen, d]`` (None: none).  `weights` ``[B, Hkv,
    max_seqlen]`` fp32, where given, is added to in place.  Allocates the outputs,
    and a workspace when none is given (attn_decode_prefix_workspace_bytes says
    how large one has to be); returns ``(o, lse, workspace)``."""
    import torch
    what, bf16 = "decode_prefix", torch.bfloat16
    gpu = q.get_device()
    if stream is not None or gpu < 0 or gpu != torch._C._cuda_getDevice():
        with _elsewhere(what, gpu, stream):
            got = decode_prefix(q, kprefix, vprefix, kcache, vcache, seqlens, scale, weights, workspace, with_lse)
        _lend(stream, q, kprefix, vprefix, kcache, vcache, seqlens if kcache is not None else None, weights, workspace)
        return got
    if q.dim() != 3 or (kcache is not None and kcache.dim() != 4) or (kprefix is not None and kprefix.dim() != 3):
        raise AttnError(ATTN_ERR_ARG, "decode_prefix: q has to be [B, Hq, d], the prefix [Hkv, P, d], the caches "
                                      "[B, Hkv, max_seqlen, d]")
    B, Hq, d = q.shape
    P = s_max = Hkv = 0
    _fits(q, bf16, q.shape, gpu) or _refuse(what, "q", q, bf16, q.shape)
    if (kcache is None) != (vcache is None) or (kprefix is None) != (vprefix is None):
        raise AttnError(ATTN_ERR_ARG, "decode_prefix: keys and values go together")
    if kcache is not None:
        Hkv, s_max = kcache.shape[1], kcache.shape[2]
        shape = (B, Hkv, s_max, d)
        _fits(kcache, bf16, shape, gpu) or _refuse(what, "kcache", kcache, bf16, shape)
        _fits(vcache, bf16, shape, gpu) or _refuse(what, "vcache", vcache, bf16, shape)
        _fits(seqlens, torch.int32, (B,), gpu) or _refuse(what, "seqlens", seqlens, torch.int32, (B,))
    if kprefix is not None:
        Hkv, P = (Hkv or kprefix.shape[0]), kprefix.shape[1]
        shape = (Hkv, P, d)
        _fits(kprefix, bf16, shape, gpu) or _refuse(what, "kprefix", kprefix, bf16, shape)
        _fits(vprefix, bf16, shape, gpu) or _refuse(what, "vprefix", vprefix, bf16, shape)
    if weights is not None:
        shape = (B, Hkv, s_max)
        _fits(weights, torch.float32, shape, gpu) or _refuse(what, "weights", weights, torch.float32, shape)
    if workspace is None:
        nbytes = attn_decode_prefix_workspace_bytes(B, Hq, Hkv, P, d, s_max, weights is not None)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    else:
        nbytes = _held(what, workspace, gpu)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if with_lse else None
    prefix = (None, None) if kprefix is None else (kprefix.data_ptr(), vprefix.data_ptr())
    own = (None, None, None) if kcache is None else (kcache.data_ptr(), vcache.data_ptr(), seqlens.data_ptr())
    rc = lib().attn_decode_prefix(q.data_ptr(), *prefix, *own, o.data_ptr(), lse.data_ptr() if with_lse else None,
                                  None if weights is None else weights.data_ptr(), B, Hq, Hkv, P, d,
                                  d ** -0.5 if scale is None else scale, s_max, workspace.data_ptr(), nbytes,
                                  torch._C._cuda_getCurrentRawStream(gpu))
    if rc:
        check(rc, "attn_decode_prefix")
    return o, lse, workspace


def decode_weighted(q, kcache, vcache, seqlens, weights, scale=None, workspace=None, with_lse=True, stream=None):
    """A decode step that adds to `weights` what every cached key receives:
    `decode_prefix` without a prefix."""
    return decode_prefix(q, None, None, kcache, vcache, seqlens, scale, weights, workspace, with_lse, stream)


def cache_evict(kcache, vcache, weights, seqlens, keep, recent=0, cache_pos=None, cur_pos=None, out=None,
                seqlens_out=None, workspace=None, stream=None):
    """Keep `keep` keys of every head's cache ``[B, Hkv, max_seqlen, d]`` by
    attn_cache_evict: the `recent` latest, then the heaviest by `weights` ``[B,
    Hkv, max_seqlen]`` fp32.  In place, unless `out` is a dict of tensors to
    write instead: ``kcache`` and ``vcache`` ``[B, Hkv, slots, d]``, optionally
    ``weights``, ``cache_pos`` ``[B, Hkv, slots]`` and ``seqlens``.  Allocates
    the new lengths and the workspace where they are not given; returns
    ``(seqlens_out, workspace)`` (`workspace` is None where none is needed)."""
    import torch
    what, bf16, i32, f32 = "cache_evict", torch.bfloat16, torch.int32, torch.float32
    gpu = kcache.get_device()
    if stream is not None or gpu < 0 or gpu != torch._C._cuda_getDevice():
        with _elsewhere(what, gpu, stream):
            got = cache_evict(kcache, vcache, weights, seqlens, keep, recent, cache_pos, cur_pos, out, seqlens_out,
                              workspace)
        _lend(stream, kcache, vcache, weights, seqlens, cache_pos, cur_pos, seqlens_out, workspace,
              *(out.values() if out is not None else ()))
        return got
    if kcache.dim() != 4:
        raise AttnError(ATTN_ERR_ARG, "cache_evict: the caches have to be [B, Hkv, max_seqlen, d]")
    B, Hkv, s_max, d = kcache.shape
    cache, per_key = kcache.shape, (B, Hkv, s_max)
    _fits(kcache, bf16, cache, gpu) or _refuse(what, "kcache", kcache, bf16, cache)
    _fits(vcache, bf16, cache, gpu) or _refuse(what, "vcache", vcache, bf16, cache)
    _fits(weights, f32, per_key, gpu) or _refuse(what, "weights", weights, f32, per_key)
    _fits(seqlens, i32, (B,), gpu) or _refuse(what, "seqlens", seqlens, i32, (B,))
    cache_pos is None or _fits(cache_pos, i32, per_key, gpu) or _refuse(what, "cache_pos", cache_pos, i32, per_key)
    cur_pos is None or _fits(cur_pos, i32, (B,), gpu) or _refuse(what, "cur_pos", cur_pos, i32, (B,))
    kout, vout, wout, pout, s_out = kcache, vcache, weights, cache_pos, s_max
    if out is not None:
        kout, vout, wout, pout = out["kcache"], out["vcache"], out.get("weights"), out.get("cache_pos")
        if seqlens_out is None:
            seqlens_out = out.get("seqlens")
        if kout.dim() != 4:
            raise AttnError(ATTN_ERR_ARG, "cache_evict: out's caches have to be [B, Hkv, slots, d]")
        s_out = kout.shape[2]
        shape, per_slot = (B, Hkv, s_out, d), (B, Hkv, s_out)
        _fits(kout, bf16, shape, gpu) or _refuse(what, "out's kcache", kout, bf16, shape)
        _fits(vout, bf16, shape, gpu) or _refuse(what, "out's vcache", vout, bf16, shape)
        wout is None or _fits(wout, f32, per_slot, gpu) or _refuse(what, "out's weights", wout, f32, per_slot)
        pout is None or _fits(pout, i32, per_slot, gpu) or _refuse(what, "out's cache_pos", pout, i32, per_slot)
    if seqlens_out is None:
        seqlens_out = torch.empty_like(seqlens)
    else:
        _fits(seqlens_out, i32, (B,), gpu) or _refuse(what, "seqlens_out", seqlens_out, i32, (B,))
    if workspace is not None:
        nbytes = _held(what, workspace, gpu)
    else:
        nbytes = attn_cache_evict_workspace_bytes(B, Hkv, s_max, keep, kout.data_ptr() == kcache.data_ptr())
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=kcache.device)
    rc = lib().attn_cache_evict(kcache.data_ptr(), vcache.data_ptr(), weights.data_ptr(),
                                None if cache_pos is None else cache_pos.data_ptr(), seqlens.data_ptr(),
                                None if cur_pos is None else cur_pos.data_ptr(), kout.data_ptr(), vout.data_ptr(),
                                None if wout is None else wout.data_ptr(), None if pout is None else pout.data_ptr(),
                                seqlens_out.data_ptr(), B, Hkv, d, s_max, s_out, keep, recent,
                                None if workspace is None else workspace.data_ptr(), nbytes,
                                torch._C._cuda_getCurrentRawStream(gpu))
    if rc:
        check(rc, "attn_cache_evict")
    return seqlens_out, workspace


def forward(q, k, v, causal=False, scale=None, tile_order=ORDER_HEAD_FIRST, with_lse=True,
            stream=None):
    """Allocate outputs and run attn_fwd_ex on ``[B, H, N, d]`` bf16 CUDA tensors."""
    import torch
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    if scale is None:
        scale = d ** -0.5
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if with_lse else None
    check(attn_fwd_ex(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, causal, tile_order, stream),
          "attn_fwd_ex")
    return o, lse


def forward_host(q, k, v, causal=False, scale=None, tile_order=ORDER_HEAD_FIRST, with_lse=True,
                 kv_heads_per_chunk=0, workspace=None, out=None, device=None, stream=None, synchronize=True):
    """Run attn_fwd_host on ``[B, H, N, d]`` bf16 CPU tensors (pinned for overlap).

    Allocates pinned outputs (unless ``out = (o, lse)`` is given) and a device
    workspace (unless given); with ``synchronize`` it waits for the stream, so
    the outputs are ready on return.  Returns ``(o, lse)``."""
    import torch
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    if scale is None:
        scale = d ** -0.5
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    nbytes = attn_fwd_host_workspace_bytes(B, Hq, Hkv, N, d, kv_heads_per_chunk)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    if out is None:
        o = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
        lse = torch.empty((B, Hq, N), dtype=torch.float32, pin_memory=True) if with_lse else None
    else:
        o, lse = out
    check(attn_fwd_host(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, causal, tile_order, kv_heads_per_chunk,
                        workspace, nbytes, stream), "attn_fwd_host")
    if synchronize:
        torch.cuda.current_stream(dev).synchronize() if stream is None else torch.cuda.synchronize(dev)
    return o, lse


def backward(q, k, v, o, lse, dout, causal=False, scale=None, tile_order=ORDER_HEAD_FIRST, workspace=None,
             stream=None):
    """Allocate gradients (and a workspace when none is given) and run attn_bwd
    on ``[B, H, N, d]`` bf16 CUDA tensors; returns ``(dq, dk, dv)``."""
    import torch
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    if scale is None:
        scale = d ** -0.5
    nbytes = attn_bwd_workspace_bytes_ex(B, Hq, Hkv, N, d, causal)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    else:
        nbytes = min(nbytes, workspace.numel() * workspace.element_size())
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    check(attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, causal, tile_order,
                   workspace, nbytes, stream), "attn_bwd")
    return dq, dk, dv


def decode(q, kcache, vcache, seqlens, num_splits=0, scale=None, workspace=None, stream=None):
    """Allocate the output (and a workspace when none is given) and run attn_decode."""
    import torch
    B, Hq, d = q.shape
    Hkv, s_max = kcache.shape[1], kcache.shape[2]
    if scale is None:
        scale = d ** -0.5
    splits = num_splits if num_splits > 0 else attn_decode_num_splits(B, Hq, Hkv, s_max)
    nbytes = attn_decode_workspace_bytes(B, Hq, d, splits)
    if workspace is None and nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    check(attn_decode(q, kcache, vcache, seqlens, o, B, Hq, Hkv, d, scale, splits, s_max,
                      workspace, nbytes, stream), "attn_decode")
    return o, workspace, splits
