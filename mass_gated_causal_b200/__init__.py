"""Python binding of the MALA C ABI (include/mala.h): argument marshalling only.

Every step of the computation runs in the sm_100a kernels of ``libmala.so``;
this module only turns torch tensors into device pointers, allocates outputs
with torch and passes the current CUDA stream. There is no CPU fallback: if the
library is missing, importing this package raises.

Raw entry points keep the C names (``mala_fwd``, ``mala_prefill``, ``mala_fwd_varlen``,
``mala_bwd``, ``mala_bwd_varlen``, ``mala_decode``, ``mala_decode_paged``, ...).
``forward``, ``prefill``, ``forward_varlen``, ``backward``, ``backward_varlen``,
``decode`` and ``decode_paged`` are conveniences that allocate the outputs and
workspaces, and so are the calls beside attention that a bounded cache needs:
``rope``, ``rope_backward``, ``rope_append``, ``key_mass``, ``key_mass_varlen``,
``decode_paged_mass``, ``evict_select``, ``evict_gather`` and ``evict``. These
also check their tensors (device, type, layout) and raise ValueError, and with
``stream`` given they allocate on that stream.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmala.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"MALA CUDA library not built: {LIB_PATH} is missing "
        "(run `python mass_gated_causal_b200/build.py` or __graft_entry__.build())")

_lib = ctypes.CDLL(LIB_PATH)

MALA_OK = 0
MALA_ERR_INVALID_ARG = 1
MALA_ERR_UNSUPPORTED = 2
MALA_ERR_WORKSPACE = 3
MALA_ERR_CUDA = 4
MALA_ERR_DEVICE_TIMEOUT = 5
MALA_ERR_RANGE = 6
MALA_FWD_PREFETCH_V = 1
MALA_ROPE_ADJACENT = 1
MALA_ROPE_CYCLIC = 2
MALA_ROPE_INVERSE = 4

EXPORTED = ("mala_status_string", "mala_abi_version", "mala_fwd", "mala_fwd_ex", "mala_prefill", "mala_fwd_varlen",
            "mala_fwd_workspace_size", "mala_bwd_workspace_size", "mala_bwd", "mala_bwd_varlen",
            "mala_decode_workspace_size", "mala_decode_default_splits", "mala_decode", "mala_decode_paged",
            "mala_decode_exact_workspace_size", "mala_decode_exact",
            "mala_decode_noalloc_max_bytes", "mala_decode_noalloc", "mala_rope", "mala_rope_append",
            "mala_key_mass_workspace_size", "mala_key_mass_varlen_workspace_size", "mala_key_mass",
            "mala_key_mass_varlen", "mala_decode_mass_workspace_size", "mala_decode_paged_mass", "mala_evict_select",
            "mala_evict_gather", "mala_test_hooks", "mala_check_status")

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_lib.mala_status_string.argtypes = [_i]
_lib.mala_status_string.restype = ctypes.c_char_p
_lib.mala_abi_version.restype = _i
_lib.mala_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _i, _i, _vp, _sz, _vp, _vp, _vp]
_lib.mala_fwd.restype = _i
_lib.mala_fwd_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _i, _i, _vp, _sz, _vp, _vp, _vp,
                             ctypes.c_uint]
_lib.mala_fwd_ex.restype = _i
_lib.mala_prefill.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _f, _i, _i, _vp, _sz, _vp, _vp,
                              _vp]
_lib.mala_prefill.restype = _i
_lib.mala_fwd_varlen.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _f, _f, _i, _i,
                                 _vp, _sz, _vp, _vp, _vp]
_lib.mala_fwd_varlen.restype = _i
_lib.mala_bwd_varlen.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _f,
                                 _i, _i, _vp, _sz, _vp, _vp, _vp]
_lib.mala_bwd_varlen.restype = _i
_lib.mala_decode_paged.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _f, _i, _vp,
                                   _sz, _vp, _vp, _vp]
_lib.mala_decode_paged.restype = _i
_lib.mala_decode_exact_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i]
_lib.mala_decode_exact_workspace_size.restype = _sz
_lib.mala_decode_exact.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _i, _i, _vp, _sz, _vp, _vp,
                                   _vp]
_lib.mala_decode_exact.restype = _i
_lib.mala_fwd_workspace_size.argtypes = [_i, _i, _i, _i]
_lib.mala_fwd_workspace_size.restype = _sz
_lib.mala_bwd_workspace_size.argtypes = [_i, _i, _i, _i]
_lib.mala_bwd_workspace_size.restype = _sz
_lib.mala_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _i, _i,
                          _vp, _sz, _vp, _vp, _vp]
_lib.mala_bwd.restype = _i
_lib.mala_decode_workspace_size.argtypes = [_i, _i, _i, _i]
_lib.mala_decode_workspace_size.restype = _sz
_lib.mala_decode_default_splits.argtypes = [_i, _i, _i, _i]
_lib.mala_decode_default_splits.restype = _i
_lib.mala_decode.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _i, _i, _vp, _sz, _vp, _vp,
                             _vp]
_lib.mala_decode.restype = _i
_lib.mala_decode_noalloc_max_bytes.restype = _sz
_lib.mala_decode_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _i, _i, _vp, _vp, _vp]
_lib.mala_decode_noalloc.restype = _i
_u = ctypes.c_uint
_lib.mala_rope.argtypes = [_vp] * 9 + [_i] * 5 + [_vp, _i, _u, _vp]
_lib.mala_rope.restype = _i
_lib.mala_rope_append.argtypes = [_vp] * 12 + [_i] * 9 + [_vp, _i, _u, _vp]
_lib.mala_rope_append.restype = _i
_lib.mala_key_mass_workspace_size.argtypes = [_i] * 6
_lib.mala_key_mass_workspace_size.restype = _sz
_lib.mala_key_mass_varlen_workspace_size.argtypes = [_i] * 7
_lib.mala_key_mass_varlen_workspace_size.restype = _sz
_lib.mala_key_mass.argtypes = [_vp] * 5 + [_i] * 6 + [_f, _i, _f, _i, _vp, _sz, _vp]
_lib.mala_key_mass.restype = _i
_lib.mala_key_mass_varlen.argtypes = [_vp] * 7 + [_i] * 8 + [_f, _i, _f, _i, _vp, _sz, _vp]
_lib.mala_key_mass_varlen.restype = _i
_lib.mala_decode_mass_workspace_size.argtypes = [_i] * 6
_lib.mala_decode_mass_workspace_size.restype = _sz
_lib.mala_decode_paged_mass.argtypes = [_vp] * 9 + [_i] * 7 + [_f, _f, _f, _i, _i, _vp, _sz, _vp, _vp, _vp]
_lib.mala_decode_paged_mass.restype = _i
_lib.mala_evict_select.argtypes = [_vp] * 5 + [_i] * 7 + [_vp]
_lib.mala_evict_select.restype = _i
_lib.mala_evict_gather.argtypes = [_vp] * 8 + [_i] * 9 + [_vp]
_lib.mala_evict_gather.restype = _i
_lib.mala_test_hooks.argtypes = [ctypes.c_ulonglong, _i, _vp]
_lib.mala_test_hooks.restype = _i
_lib.mala_check_status.argtypes = [_vp]
_lib.mala_check_status.restype = _i


class MalaError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {mala_status_string(code)} ({code})")
        self.code = code


def _p(x) -> Optional[int]:
    """Device pointer of a tensor (or pass an int / None through)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str) -> None:
    if rc != MALA_OK:
        raise MalaError(rc, where)


# ------------------------------------------------------------- raw C names
def mala_status_string(code: int) -> str:
    return _lib.mala_status_string(int(code)).decode()


def mala_abi_version() -> int:
    return int(_lib.mala_abi_version())


def mala_fwd(q, k, v, o, lse, B, Hq, Hkv, L, d, scale, tau, Bq, Bk, workspace, workspace_bytes, kept_tiles,
             keep_map=None, stream=None) -> int:
    return int(_lib.mala_fwd(_p(q), _p(k), _p(v), _p(o), _p(lse), B, Hq, Hkv, L, d, float(scale), float(tau),
                             Bq, Bk, _p(workspace), int(workspace_bytes), _p(kept_tiles), _p(keep_map),
                             _stream(stream)))


def mala_fwd_ex(q, k, v, o, lse, B, Hq, Hkv, L, d, scale, tau, Bq, Bk, workspace, workspace_bytes, kept_tiles,
                keep_map=None, stream=None, flags=0) -> int:
    return int(_lib.mala_fwd_ex(_p(q), _p(k), _p(v), _p(o), _p(lse), B, Hq, Hkv, L, d, float(scale), float(tau),
                                Bq, Bk, _p(workspace), int(workspace_bytes), _p(kept_tiles), _p(keep_map),
                                _stream(stream), int(flags)))


def mala_prefill(q, k, v, o, lse, B, Hq, Hkv, Lq, Lk, d, scale, tau, Bq, Bk, workspace, workspace_bytes,
                 kept_tiles, keep_map=None, stream=None) -> int:
    return int(_lib.mala_prefill(_p(q), _p(k), _p(v), _p(o), _p(lse), B, Hq, Hkv, Lq, Lk, d, float(scale),
                                 float(tau), Bq, Bk, _p(workspace), int(workspace_bytes), _p(kept_tiles),
                                 _p(keep_map), _stream(stream)))


def mala_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, num_seqs, max_seqlen_q, max_seqlen_k, total_q,
                    total_k, Hq, Hkv, d, scale, tau, Bq, Bk, workspace, workspace_bytes, kept_tiles, keep_map=None,
                    stream=None) -> int:
    return int(_lib.mala_fwd_varlen(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(cu_seqlens_q), _p(cu_seqlens_k),
                                    num_seqs, max_seqlen_q, max_seqlen_k, total_q, total_k, Hq, Hkv, d,
                                    float(scale), float(tau), Bq, Bk, _p(workspace), int(workspace_bytes),
                                    _p(kept_tiles), _p(keep_map), _stream(stream)))


def mala_bwd_varlen(q, k, v, o, do, lse, dq, dk, dv, cu_seqlens, num_seqs, max_seqlen, total, Hq, Hkv, d, scale,
                    tau, Bq, Bk, workspace, workspace_bytes, kept_tiles, keep_map=None, stream=None) -> int:
    return int(_lib.mala_bwd_varlen(_p(q), _p(k), _p(v), _p(o), _p(do), _p(lse), _p(dq), _p(dk), _p(dv),
                                    _p(cu_seqlens), num_seqs, max_seqlen, total, Hq, Hkv, d, float(scale),
                                    float(tau), Bq, Bk, _p(workspace), int(workspace_bytes), _p(kept_tiles),
                                    _p(keep_map), _stream(stream)))


def mala_decode_paged(q, k_pages, v_pages, block_table, seqlens_k, o, lse, B, Hq, Hkv, num_pages, page_size,
                      max_pages_per_seq, d, scale, tau, n_splits, workspace, workspace_bytes, kept_tiles,
                      keep_map=None, stream=None) -> int:
    return int(_lib.mala_decode_paged(_p(q), _p(k_pages), _p(v_pages), _p(block_table), _p(seqlens_k), _p(o),
                                      _p(lse), B, Hq, Hkv, num_pages, page_size, max_pages_per_seq, d,
                                      float(scale), float(tau), n_splits, _p(workspace), int(workspace_bytes),
                                      _p(kept_tiles), _p(keep_map), _stream(stream)))


def mala_fwd_workspace_size(B, Hkv, L, d) -> int:
    return int(_lib.mala_fwd_workspace_size(B, Hkv, L, d))


def mala_bwd_workspace_size(B, Hq, L, d) -> int:
    return int(_lib.mala_bwd_workspace_size(B, Hq, L, d))


def mala_bwd(q, k, v, o, do, lse, dq, dk, dv, B, Hq, Hkv, L, d, scale, tau, Bq, Bk, workspace, workspace_bytes,
             kept_tiles, keep_map=None, stream=None) -> int:
    return int(_lib.mala_bwd(_p(q), _p(k), _p(v), _p(o), _p(do), _p(lse), _p(dq), _p(dk), _p(dv), B, Hq, Hkv, L,
                             d, float(scale), float(tau), Bq, Bk, _p(workspace), int(workspace_bytes),
                             _p(kept_tiles), _p(keep_map), _stream(stream)))


def mala_decode_workspace_size(B, Hq, d, n_splits) -> int:
    return int(_lib.mala_decode_workspace_size(B, Hq, d, n_splits))


def mala_decode_default_splits(B, Hkv, Lk, Bk) -> int:
    return int(_lib.mala_decode_default_splits(B, Hkv, Lk, Bk))


def mala_decode(q, kcache, vcache, o, lse, B, Hq, Hkv, Lk, d, scale, tau, Bk, n_splits, workspace,
                workspace_bytes, kept_tiles, keep_map=None, stream=None) -> int:
    return int(_lib.mala_decode(_p(q), _p(kcache), _p(vcache), _p(o), _p(lse), B, Hq, Hkv, Lk, d, float(scale),
                                float(tau), Bk, n_splits, _p(workspace), int(workspace_bytes), _p(kept_tiles),
                                _p(keep_map), _stream(stream)))


def mala_decode_exact_workspace_size(B, Hq, Lk, d, Bk, n_splits) -> int:
    return int(_lib.mala_decode_exact_workspace_size(B, Hq, Lk, d, Bk, n_splits))


def mala_decode_exact(q, kcache, vcache, o, lse, B, Hq, Hkv, Lk, d, scale, tau, Bk, n_splits, workspace,
                      workspace_bytes, kept_tiles, keep_map=None, stream=None) -> int:
    return int(_lib.mala_decode_exact(_p(q), _p(kcache), _p(vcache), _p(o), _p(lse), B, Hq, Hkv, Lk, d,
                                      float(scale), float(tau), Bk, n_splits, _p(workspace), int(workspace_bytes),
                                      _p(kept_tiles), _p(keep_map), _stream(stream)))


def mala_decode_noalloc_max_bytes() -> int:
    return int(_lib.mala_decode_noalloc_max_bytes())


def mala_decode_noalloc(q, kcache, vcache, o, lse, B, Hq, Hkv, Lk, d, scale, tau, Bk, n_splits, kept_tiles,
                        keep_map=None, stream=None) -> int:
    return int(_lib.mala_decode_noalloc(_p(q), _p(kcache), _p(vcache), _p(o), _p(lse), B, Hq, Hkv, Lk, d,
                                        float(scale), float(tau), Bk, n_splits, _p(kept_tiles), _p(keep_map),
                                        _stream(stream)))


def _host_array(values, ctype):
    """A HOST array argument (None passes through)."""
    return None if values is None else (ctype * len(values))(*values)


def mala_rope(q, k, v, q_out, k_out, v_out, strides, positions, inv_freq, T, Hq, Hkv, d, rotary_dim, sections, n_axes,
              flags=0, stream=None) -> int:
    """strides: 12 ints, sections: n_axes ints (host sequences)."""
    return int(_lib.mala_rope(_p(q), _p(k), _p(v), _p(q_out), _p(k_out), _p(v_out),
                              _host_array(strides, ctypes.c_int64), _p(positions), _p(inv_freq), T, Hq, Hkv, d,
                              rotary_dim, _host_array(sections, ctypes.c_int32), n_axes, flags, _stream(stream)))


def mala_rope_append(q, k, v, q_out, strides, positions, inv_freq, k_pages, v_pages, block_table, seqlens_k,
                     cu_seqlens, num_seqs, T, Hq, Hkv, num_pages, page_size, max_pages_per_seq, d, rotary_dim,
                     sections, n_axes, flags=0, stream=None) -> int:
    """strides: 8 ints, sections: n_axes ints (host sequences)."""
    return int(_lib.mala_rope_append(_p(q), _p(k), _p(v), _p(q_out), _host_array(strides, ctypes.c_int64),
                                     _p(positions), _p(inv_freq), _p(k_pages), _p(v_pages), _p(block_table),
                                     _p(seqlens_k), _p(cu_seqlens), num_seqs, T, Hq, Hkv, num_pages, page_size,
                                     max_pages_per_seq, d, rotary_dim, _host_array(sections, ctypes.c_int32), n_axes,
                                     flags, _stream(stream)))


def mala_key_mass_workspace_size(B, Hq, Hkv, Lq, Lk, window) -> int:
    return int(_lib.mala_key_mass_workspace_size(B, Hq, Hkv, Lq, Lk, window))


def mala_key_mass_varlen_workspace_size(num_seqs, Hq, Hkv, max_seqlen_q, max_seqlen_k, total_q, window) -> int:
    return int(_lib.mala_key_mass_varlen_workspace_size(num_seqs, Hq, Hkv, max_seqlen_q, max_seqlen_k, total_q,
                                                        window))


def mala_key_mass(q, k, lse, mass_in, mass_out, B, Hq, Hkv, Lq, Lk, d, scale, window, decay, ld_mass, workspace,
                  workspace_bytes, stream=None) -> int:
    return int(_lib.mala_key_mass(_p(q), _p(k), _p(lse), _p(mass_in), _p(mass_out), B, Hq, Hkv, Lq, Lk, d,
                                  float(scale), window, float(decay), ld_mass, _p(workspace), int(workspace_bytes),
                                  _stream(stream)))


def mala_key_mass_varlen(q, k, lse, cu_seqlens_q, cu_seqlens_k, mass_in, mass_out, num_seqs, max_seqlen_q,
                         max_seqlen_k, total_q, total_k, Hq, Hkv, d, scale, window, decay, ld_mass, workspace,
                         workspace_bytes, stream=None) -> int:
    return int(_lib.mala_key_mass_varlen(_p(q), _p(k), _p(lse), _p(cu_seqlens_q), _p(cu_seqlens_k), _p(mass_in),
                                         _p(mass_out), num_seqs, max_seqlen_q, max_seqlen_k, total_q, total_k, Hq,
                                         Hkv, d, float(scale), window, float(decay), ld_mass, _p(workspace),
                                         int(workspace_bytes), _stream(stream)))


def mala_decode_mass_workspace_size(B, Hq, d, page_size, max_pages_per_seq, n_splits) -> int:
    return int(_lib.mala_decode_mass_workspace_size(B, Hq, d, page_size, max_pages_per_seq, n_splits))


def mala_decode_paged_mass(q, k_pages, v_pages, block_table, seqlens_k, o, lse, mass_in, mass_out, B, Hq, Hkv,
                           num_pages, page_size, max_pages_per_seq, d, scale, tau, decay, ld_mass, n_splits, workspace,
                           workspace_bytes, kept_tiles, keep_map=None, stream=None) -> int:
    return int(_lib.mala_decode_paged_mass(_p(q), _p(k_pages), _p(v_pages), _p(block_table), _p(seqlens_k), _p(o),
                                           _p(lse), _p(mass_in), _p(mass_out), B, Hq, Hkv, num_pages, page_size,
                                           max_pages_per_seq, d, float(scale), float(tau), float(decay), ld_mass,
                                           n_splits, _p(workspace), int(workspace_bytes), _p(kept_tiles),
                                           _p(keep_map), _stream(stream)))


def mala_evict_select(mass, seqlens_k, index, new_seqlens, mass_out, B, Hkv, ld_mass, budget, n_sink, n_recent,
                      ld_mass_out, stream=None) -> int:
    return int(_lib.mala_evict_select(_p(mass), _p(seqlens_k), _p(index), _p(new_seqlens), _p(mass_out), B, Hkv,
                                      ld_mass, budget, n_sink, n_recent, ld_mass_out, _stream(stream)))


def mala_evict_gather(k_pages, v_pages, block_table, index, new_seqlens, k_out_pages, v_out_pages, out_table, B, Hkv,
                      budget, num_pages, num_out_pages, page_size, max_pages_per_seq, max_out_pages_per_seq, d,
                      stream=None) -> int:
    return int(_lib.mala_evict_gather(_p(k_pages), _p(v_pages), _p(block_table), _p(index), _p(new_seqlens),
                                      _p(k_out_pages), _p(v_out_pages), _p(out_table), B, Hkv, budget, num_pages,
                                      num_out_pages, page_size, max_pages_per_seq, max_out_pages_per_seq, d,
                                      _stream(stream)))


def mala_test_hooks(wait_limit_ns: int = 0, stall_tile: int = -1, fwd_v_tiles=None) -> int:
    return int(_lib.mala_test_hooks(int(wait_limit_ns), int(stall_tile), _p(fwd_v_tiles)))


def mala_check_status(stream=None) -> int:
    return int(_lib.mala_check_status(_stream(stream)))


# ------------------------------------------------------------ conveniences
def forward(q, k, v, scale: float, tau: float, Bq: int = 128, Bk: int = 128, keep_map: bool = False,
            workspace=None, stream=None, prefetch_v: bool = False):
    """q [B,L,Hq,d], k/v [B,L,Hkv,d] bf16 CUDA tensors -> (o, lse, kept_tiles, keep_map|None).

    prefetch_v: fetch every V tile ahead of the gate (mala_fwd_ex with MALA_FWD_PREFETCH_V)."""
    import torch
    B, L, Hq, d = q.shape
    Hkv = k.shape[2]
    if workspace is None:
        workspace = torch.empty((max(1, mala_fwd_workspace_size(B, Hkv, L, d)),), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, L), dtype=torch.float32, device=q.device)
    kept = torch.empty((B * Hq,), dtype=torch.int32, device=q.device)
    km = None
    if keep_map:
        km = torch.full((B, Hq, -(-L // Bq), -(-L // Bk)), 255, dtype=torch.uint8, device=q.device)
    _check(mala_fwd_ex(q, k, v, o, lse, B, Hq, Hkv, L, d, scale, tau, Bq, Bk, workspace,
                       workspace.numel() * workspace.element_size(), kept, km, stream,
                       MALA_FWD_PREFETCH_V if prefetch_v else 0), "mala_fwd")
    return o, lse, kept, km


def prefill(q, k, v, scale: float, tau: float, Bq: int = 128, Bk: int = 128, keep_map: bool = False,
            workspace=None, stream=None):
    """q [B,Lq,Hq,d] (new queries), k/v [B,Lk,Hkv,d] (cache incl. the new keys)
    -> (o [B,Lq,Hq,d], lse [B,Hq,Lq], kept_tiles, keep_map|None)."""
    import torch
    B, Lq, Hq, d = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    if workspace is None:
        workspace = torch.empty((max(1, mala_fwd_workspace_size(B, Hkv, Lk, d)),), dtype=torch.uint8,
                                device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    kept = torch.empty((B * Hq,), dtype=torch.int32, device=q.device)
    km = None
    if keep_map:
        km = torch.full((B, Hq, -(-Lq // Bq), -(-Lk // Bk)), 255, dtype=torch.uint8, device=q.device)
    _check(mala_prefill(q, k, v, o, lse, B, Hq, Hkv, Lq, Lk, d, scale, tau, Bq, Bk, workspace,
                        workspace.numel() * workspace.element_size(), kept, km, stream), "mala_prefill")
    return o, lse, kept, km


def forward_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int, scale: float,
                   tau: float, Bq: int = 128, Bk: int = 128, keep_map: bool = False, workspace=None, stream=None):
    """Packed batch: q [total_q,Hq,d], k/v [total_k,Hkv,d] bf16; cu_seqlens_* int32 CUDA tensors
    [num_seqs+1] -> (o [total_q,Hq,d], lse [Hq,total_q], kept_tiles [num_seqs*Hq], keep_map|None)."""
    import torch
    total_q, Hq, d = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    S = cu_seqlens_q.numel() - 1
    if workspace is None:
        workspace = torch.empty((max(1, mala_fwd_workspace_size(1, Hkv, total_k, d)),), dtype=torch.uint8,
                                device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device)
    kept = torch.empty((S * Hq,), dtype=torch.int32, device=q.device)
    km = None
    if keep_map:
        km = torch.full((S, Hq, -(-max_seqlen_q // Bq), -(-max_seqlen_k // Bk)), 255, dtype=torch.uint8,
                        device=q.device)
    _check(mala_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, S, max_seqlen_q, max_seqlen_k, total_q,
                           total_k, Hq, Hkv, d, scale, tau, Bq, Bk, workspace,
                           workspace.numel() * workspace.element_size(), kept, km, stream), "mala_fwd_varlen")
    return o, lse, kept, km


def backward_varlen(q, k, v, o, do, lse, cu_seqlens, max_seqlen: int, scale: float, tau: float, Bq: int = 128,
                    Bk: int = 128, keep_map: bool = False, workspace=None, stream=None):
    """Packed training batch -> (dq, dk, dv, kept_tiles [num_seqs*Hq], keep_map|None)."""
    import torch
    total, Hq, d = q.shape
    Hkv = k.shape[1]
    S = cu_seqlens.numel() - 1
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    kept = torch.empty((S * Hq,), dtype=torch.int32, device=q.device)
    if workspace is None:
        workspace = torch.empty((mala_bwd_workspace_size(1, Hq, total, d),), dtype=torch.uint8, device=q.device)
    km = None
    if keep_map:
        km = torch.full((S, Hq, -(-max_seqlen // Bq), -(-max_seqlen // Bk)), 255, dtype=torch.uint8,
                        device=q.device)
    _check(mala_bwd_varlen(q, k, v, o, do, lse, dq, dk, dv, cu_seqlens, S, max_seqlen, total, Hq, Hkv, d, scale,
                           tau, Bq, Bk, workspace, workspace.numel() * workspace.element_size(), kept, km,
                           stream), "mala_bwd_varlen")
    return dq, dk, dv, kept, km


def backward(q, k, v, o, do, lse, scale: float, tau: float, Bq: int = 128, Bk: int = 128,
             keep_map: bool = False, workspace=None, stream=None):
    """-> (dq, dk, dv, kept_tiles, keep_map|None)."""
    import torch
    B, L, Hq, d = q.shape
    Hkv = k.shape[2]
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    kept = torch.empty((B * Hq,), dtype=torch.int32, device=q.device)
    ws_bytes = mala_bwd_workspace_size(B, Hq, L, d)
    if workspace is None:
        workspace = torch.empty((ws_bytes,), dtype=torch.uint8, device=q.device)
    km = None
    if keep_map:
        km = torch.full((B, Hq, -(-L // Bq), -(-L // Bk)), 255, dtype=torch.uint8, device=q.device)
    _check(mala_bwd(q, k, v, o, do, lse, dq, dk, dv, B, Hq, Hkv, L, d, scale, tau, Bq, Bk, workspace,
                    workspace.numel() * workspace.element_size(), kept, km, stream), "mala_bwd")
    return dq, dk, dv, kept, km


def decode(q, kcache, vcache, scale: float, tau: float, Bk: int = 128, n_splits: int = 0,
           keep_map: bool = False, workspace=None, stream=None):
    """q [B,Hq,d], kcache/vcache [B,Lk,Hkv,d] -> (o, lse, kept_tiles, keep_map|None, n_splits)."""
    import torch
    B, Hq, d = q.shape
    Lk, Hkv = kcache.shape[1], kcache.shape[2]
    if n_splits == 0:
        n_splits = mala_decode_default_splits(B, Hkv, Lk, Bk)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    kept = torch.empty((B * Hq,), dtype=torch.int32, device=q.device)
    ws_bytes = mala_decode_workspace_size(B, Hq, d, n_splits)
    if workspace is None:
        workspace = torch.empty((max(ws_bytes, 1),), dtype=torch.uint8, device=q.device)
    km = torch.full((B, Hq, -(-Lk // Bk)), 255, dtype=torch.uint8, device=q.device) if keep_map else None
    _check(mala_decode(q, kcache, vcache, o, lse, B, Hq, Hkv, Lk, d, scale, tau, Bk, n_splits, workspace,
                       workspace.numel() * workspace.element_size(), kept, km, stream), "mala_decode")
    return o, lse, kept, km, n_splits


def decode_paged(q, k_pages, v_pages, block_table, seqlens_k, scale: float, tau: float, n_splits: int = 0,
                 keep_map: bool = False, workspace=None, stream=None):
    """q [B,Hq,d]; k_pages/v_pages [num_pages,page,Hkv,d]; block_table [B,max_pages] and
    seqlens_k [B] int32 CUDA tensors -> (o, lse, kept_tiles, keep_map|None, n_splits)."""
    import torch
    B, Hq, d = q.shape
    num_pages, page, Hkv = k_pages.shape[0], k_pages.shape[1], k_pages.shape[2]
    maxp = block_table.shape[1]
    if n_splits == 0:
        n_splits = mala_decode_default_splits(B, Hkv, maxp * page, page)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    kept = torch.empty((B * Hq,), dtype=torch.int32, device=q.device)
    ws_bytes = mala_decode_workspace_size(B, Hq, d, n_splits)
    if workspace is None:
        workspace = torch.empty((max(ws_bytes, 1),), dtype=torch.uint8, device=q.device)
    km = torch.full((B, Hq, maxp), 255, dtype=torch.uint8, device=q.device) if keep_map else None
    _check(mala_decode_paged(q, k_pages, v_pages, block_table, seqlens_k, o, lse, B, Hq, Hkv, num_pages, page, maxp,
                             d, scale, tau, n_splits, workspace, workspace.numel() * workspace.element_size(), kept,
                             km, stream), "mala_decode_paged")
    return o, lse, kept, km, n_splits


def decode_exact(q, kcache, vcache, scale: float, tau: float, Bk: int = 128, n_splits: int = 0,
                 keep_map: bool = False, workspace=None, stream=None):
    """Split-independent decode -> (o, lse, kept_tiles, keep_map|None, n_splits)."""
    import torch
    B, Hq, d = q.shape
    Lk, Hkv = kcache.shape[1], kcache.shape[2]
    if n_splits == 0:
        n_splits = mala_decode_default_splits(B, Hkv, Lk, Bk)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    kept = torch.empty((B * Hq,), dtype=torch.int32, device=q.device)
    ws_bytes = mala_decode_exact_workspace_size(B, Hq, Lk, d, Bk, n_splits)
    if workspace is None:
        workspace = torch.empty((max(ws_bytes, 1),), dtype=torch.uint8, device=q.device)
    km = torch.full((B, Hq, -(-Lk // Bk)), 255, dtype=torch.uint8, device=q.device) if keep_map else None
    _check(mala_decode_exact(q, kcache, vcache, o, lse, B, Hq, Hkv, Lk, d, scale, tau, Bk, n_splits, workspace,
                             workspace.numel() * workspace.element_size(), kept, km, stream), "mala_decode_exact")
    return o, lse, kept, km, n_splits


# ------------------------------------------------- beside attention: positions, masses, eviction
# Their calls are short (a decoding step's rotation takes a few microseconds on the GPU), so the
# checks below are kept cheap: one comparison per property, names and messages only on a failure.
def _device(where, x) -> int:
    """The current device's index, which the call's tensors must be on."""
    import torch
    dev = torch.cuda.current_device() if x.is_cuda else -1
    if x.get_device() != dev or dev < 0:
        raise ValueError(f"{where}: tensors must be on the current CUDA device, got {x.device}")
    return dev


def _need(where, dtype, dev, contiguous, *tensors) -> None:
    """Every tensor given (None: left out) has this type, is on this device and, if asked, contiguous."""
    for x in tensors:
        if x is not None and (x.dtype is not dtype or x.get_device() != dev or
                              (contiguous and not x.is_contiguous())):
            raise ValueError(f"{where}: expected a {'contiguous ' if contiguous else ''}{dtype} tensor on device {dev}, "
                             f"got {x.dtype} {tuple(x.shape)} with strides {x.stride()} on {x.device}")


def _shape(where, name, x, *shape) -> None:
    if x is not None and x.shape != shape:
        raise ValueError(f"{where}: {name} must have shape {shape}, got {tuple(x.shape)}")


def _rows(where, name, x):
    """(tokens, heads, d, token stride, head stride) of a tensor [..., H, d] whose leading axes
    step through its tokens with one stride."""
    shape, stride = x.shape, x.stride()
    if len(shape) < 3 or stride[-1] != 1:
        raise ValueError(f"{where}: {name} must be [..., H, d] with adjacent values in a head")
    if len(shape) == 3:
        tokens, step = shape[0], stride[0]
    else:
        tokens, step = 1, 0
        for n, st in zip(shape[-3::-1], stride[-3::-1]):
            if n == 1:
                continue
            if tokens == 1:
                step = st
            elif st != step * tokens:
                raise ValueError(f"{where}: the tokens of {name} must lie at one stride")
            tokens *= n
    # the stride of an axis with one entry means nothing
    return tokens, shape[-2], shape[-1], step if tokens > 1 else 0, stride[-2] if shape[-2] > 1 else 0


def _on(stream):
    """Allocate on the stream the call runs on (torch orders a block's reuse by that stream)."""
    import torch
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _empty(shape, dtype, dev, stream):
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _raw_stream(stream, dev) -> int:
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


_I64x12, _I64x8 = ctypes.c_int64 * 12, ctypes.c_int64 * 8


@functools.lru_cache(maxsize=256)
def _sections(sections):
    return (ctypes.c_int32 * len(sections))(*sections), len(sections)


def _rope_tables(where, positions, inv_freq, sections, T, dev):
    import torch
    _need(where, torch.int32, dev, True, positions)
    _need(where, torch.float32, dev, True, inv_freq)
    pairs = inv_freq.numel()
    arr, n_axes = _sections((pairs,) if sections is None else tuple(sections))
    if positions.numel() != n_axes * T:
        raise ValueError(f"{where}: positions must be [{n_axes}, {T}], got {tuple(positions.shape)}")
    return arr, n_axes, 2 * pairs


def _rope_call(where, q, k, v, positions, inv_freq, sections, flags, out, stream):
    import torch
    first = q if q is not None else k if k is not None else v
    if first is None:
        raise ValueError(f"{where}: no tensor given")
    dev = _device(where, first)
    _need(where, torch.bfloat16, dev, False, q, k, v)
    if out is None:
        out = tuple(None if x is None else _empty(x.shape, x.dtype, dev, stream) for x in (q, k, v))
    else:
        _need(where, torch.bfloat16, dev, False, *out)
    T = d = None
    heads = [1, 1, 1]
    ptrs, strides = [None] * 6, [0] * 12
    for w, x, y in zip((0, 1, 2), (q, k, v), out):
        if x is None and y is None:
            continue
        if x is None or y is None:
            raise ValueError(f"{where}: {'qkv'[w]} needs both its input and its output")
        n, h, dx, st, sh = _rows(where, "qkv"[w], x)
        if y.shape != x.shape and _rows(where, "out", y)[:3] != (n, h, dx):
            raise ValueError(f"{where}: {'qkv'[w]} and its output disagree in shape")
        if T is None:
            T, d = n, dx
        elif (n, dx) != (T, d):
            raise ValueError(f"{where}: q, k and v disagree in tokens or head size")
        heads[w] = h
        ptrs[w], ptrs[3 + w] = x.data_ptr(), y.data_ptr()
        strides[2 * w:2 * w + 2] = st, sh
        strides[6 + 2 * w:8 + 2 * w] = _rows(where, "out", y)[3:]
    if k is not None and v is not None and heads[1] != heads[2]:
        raise ValueError(f"{where}: k and v disagree in heads")
    arr, n_axes, rot = _rope_tables(where, positions, inv_freq, sections, T, dev)
    rc = _lib.mala_rope(*ptrs, _I64x12(*strides), positions.data_ptr(), inv_freq.data_ptr(), T, heads[0],
                        heads[1] if k is not None else heads[2], d, rot, arr, n_axes, flags, _raw_stream(stream, dev))
    if rc:
        _check(rc, where)
    return out


def _rope_flags(adjacent, cyclic):
    return (MALA_ROPE_ADJACENT if adjacent else 0) | (MALA_ROPE_CYCLIC if cyclic else 0)


def rope(q, k, v, positions, inv_freq, sections=None, adjacent: bool = False, cyclic: bool = False, out=None,
         stream=None):
    """Rotary positions: q [..., Hq, d], k and v [..., Hkv, d] bf16 (strided views of a fused projection's
    output will do; any may be None), positions [n_axes, T] or [T] int32, inv_freq [rotary_dim / 2] fp32,
    sections: pairs per axis (None: one axis) -> contiguous (q, k, v), or out = (q, k, v) to write to."""
    return _rope_call("mala_rope", q, k, v, positions, inv_freq, sections, _rope_flags(adjacent, cyclic), out, stream)


def rope_backward(dq, dk, dv, positions, inv_freq, sections=None, adjacent: bool = False, cyclic: bool = False,
                  out=None, stream=None):
    """Gradient of rope: dq, dk, dv of its outputs -> those of its inputs (out: views of a fused gradient)."""
    return _rope_call("mala_rope", dq, dk, dv, positions, inv_freq, sections,
                      _rope_flags(adjacent, cyclic) | MALA_ROPE_INVERSE, out, stream)


def rope_append(q, k, v, positions, inv_freq, k_pages, v_pages, block_table, seqlens_k, cu_seqlens=None, sections=None,
                adjacent: bool = False, cyclic: bool = False, out=None, stream=None):
    """Rotate a serving step's new tokens q [T, Hq, d], k, v [T, Hkv, d] (strided views will do; q may be None)
    and write k and v into the paged cache; seqlens_k counts the new tokens, cu_seqlens [num_seqs+1] says whose
    they are (None: T / num_seqs each) -> rotated q."""
    import torch
    where = "mala_rope_append"
    dev = _device(where, k)
    _need(where, torch.bfloat16, dev, False, q, k, v)
    _need(where, torch.bfloat16, dev, True, k_pages, v_pages)
    _need(where, torch.int32, dev, True, block_table, seqlens_k, cu_seqlens)
    T, Hkv, d, kt, kh = _rows(where, "k", k)
    Tv, Hv, dv, vt, vh = _rows(where, "v", v)
    if (Tv, Hv, dv) != (T, Hkv, d):
        raise ValueError(f"{where}: k and v disagree in tokens, heads or head size")
    pool = k_pages.shape
    S = seqlens_k.numel()
    if len(pool) != 4 or pool[2] != Hkv or pool[3] != d or v_pages.shape != pool:
        raise ValueError(f"{where}: pools must be [num_pages, page, {Hkv}, {d}], got {tuple(pool)} and "
                         f"{tuple(v_pages.shape)}")
    maxp = block_table.shape[-1]
    _shape(where, "block_table", block_table, S, maxp)
    cu = None
    if cu_seqlens is not None:
        _shape(where, "cu_seqlens", cu_seqlens, S + 1)
        cu = cu_seqlens.data_ptr()
    qp = op = None
    qt = qh = ot = oh = 0
    Hq = 1
    if q is not None:
        Tq, Hq, dq, qt, qh = _rows(where, "q", q)
        if out is None:
            out = _empty(q.shape, q.dtype, dev, stream)
        else:
            _need(where, torch.bfloat16, dev, False, out)
        To, Ho, do, ot, oh = _rows(where, "out", out)
        if (Tq, dq) != (T, d) or (To, Ho, do) != (T, Hq, d):
            raise ValueError(f"{where}: q, out and k disagree in tokens, heads or head size")
        qp, op = q.data_ptr(), out.data_ptr()
    elif out is not None:
        raise ValueError(f"{where}: out without q")
    arr, n_axes, rot = _rope_tables(where, positions, inv_freq, sections, T, dev)
    rc = _lib.mala_rope_append(qp, k.data_ptr(), v.data_ptr(), op, _I64x8(qt, qh, kt, kh, vt, vh, ot, oh),
                               positions.data_ptr(), inv_freq.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                               block_table.data_ptr(), seqlens_k.data_ptr(), cu, S, T, Hq, Hkv, pool[0], pool[1], maxp,
                               d, rot, arr, n_axes, _rope_flags(adjacent, cyclic), _raw_stream(stream, dev))
    if rc:
        _check(rc, where)
    return out


def _mass_out(where, mass, out, B, Hkv, ld, dev, stream):
    """(masses to write, their row length): the output given, or a new one as long as the input."""
    import torch
    _need(where, torch.float32, dev, True, mass, out)
    if mass is not None:
        ld = mass.shape[-1]
        _shape(where, "mass", mass, B, Hkv, ld)
    elif out is not None:
        ld = out.shape[-1]
    if out is None:
        return _empty((B, Hkv, ld), torch.float32, dev, stream), ld
    _shape(where, "out", out, B, Hkv, ld)
    return out, ld


def _scratch(where, workspace, need, dev, stream):
    """(pointer, bytes) of the workspace: the caller's, or a new one (kept by the third value)."""
    import torch
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _empty((need,), torch.uint8, dev, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"{where}: the workspace must be contiguous and on device {dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def key_mass(q, k, lse, scale: float, window: int = 0, mass=None, decay: float = 1.0, out=None, workspace=None,
             stream=None):
    """The attention weight each key collected: q [B,Lq,Hq,d], k [B,Lk,Hkv,d] bf16 and lse [B,Hq,Lq] of a forward
    or prefill call; window: only the last rows count (0: all); mass [B,Hkv,ld] fp32: what earlier calls
    collected, times decay -> mass [B,Hkv,ld] (ld = Lk unless mass or out says more; out may be mass)."""
    import torch
    where = "mala_key_mass"
    dev = _device(where, q)
    B, Lq, Hq, d = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    _need(where, torch.bfloat16, dev, True, q, k)
    _need(where, torch.float32, dev, True, lse)
    _shape(where, "k", k, B, Lk, Hkv, d)
    _shape(where, "lse", lse, B, Hq, Lq)
    out, ld = _mass_out(where, mass, out, B, Hkv, Lk, dev, stream)
    ws, ws_bytes, _hold = _scratch(where, workspace, _lib.mala_key_mass_workspace_size(B, Hq, Hkv, Lq, Lk, window),
                                   dev, stream)
    rc = _lib.mala_key_mass(q.data_ptr(), k.data_ptr(), lse.data_ptr(), None if mass is None else mass.data_ptr(),
                            out.data_ptr(), B, Hq, Hkv, Lq, Lk, d, scale, window, decay, ld, ws, ws_bytes,
                            _raw_stream(stream, dev))
    if rc:
        _check(rc, where)
    return out


def key_mass_varlen(q, k, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int, scale: float,
                    window: int = 0, mass=None, decay: float = 1.0, out=None, workspace=None, stream=None):
    """key_mass of a packed batch: q [total_q,Hq,d], k [total_k,Hkv,d], lse [Hq,total_q] as forward_varlen takes
    and leaves them -> mass [num_seqs,Hkv,ld] (ld = max_seqlen_k unless mass or out says more)."""
    import torch
    where = "mala_key_mass_varlen"
    dev = _device(where, q)
    total_q, Hq, d = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    S = cu_seqlens_q.numel() - 1
    _need(where, torch.bfloat16, dev, True, q, k)
    _need(where, torch.float32, dev, True, lse)
    _need(where, torch.int32, dev, True, cu_seqlens_q, cu_seqlens_k)
    _shape(where, "k", k, total_k, Hkv, d)
    _shape(where, "lse", lse, Hq, total_q)
    _shape(where, "cu_seqlens_k", cu_seqlens_k, S + 1)
    out, ld = _mass_out(where, mass, out, S, Hkv, max_seqlen_k, dev, stream)
    need = _lib.mala_key_mass_varlen_workspace_size(S, Hq, Hkv, max_seqlen_q, max_seqlen_k, total_q, window)
    ws, ws_bytes, _hold = _scratch(where, workspace, need, dev, stream)
    rc = _lib.mala_key_mass_varlen(q.data_ptr(), k.data_ptr(), lse.data_ptr(), cu_seqlens_q.data_ptr(),
                                   cu_seqlens_k.data_ptr(), None if mass is None else mass.data_ptr(), out.data_ptr(),
                                   S, max_seqlen_q, max_seqlen_k, total_q, total_k, Hq, Hkv, d, scale, window, decay,
                                   ld, ws, ws_bytes, _raw_stream(stream, dev))
    if rc:
        _check(rc, where)
    return out


def decode_paged_mass(q, k_pages, v_pages, block_table, seqlens_k, scale: float, tau: float, mass=None,
                      decay: float = 1.0, out=None, n_splits: int = 0, keep_map: bool = False, workspace=None,
                      stream=None):
    """decode_paged that also collects each key's weight: mass [B,Hkv,ld] fp32 of earlier calls (None: 0), ld >=
    max_pages * page -> (o, lse, kept_tiles, keep_map|None, n_splits, mass); out: where the masses go (may be mass)."""
    import torch
    where = "mala_decode_paged_mass"
    dev = _device(where, q)
    B, Hq, d = q.shape
    pool = k_pages.shape
    if len(pool) != 4 or pool[3] != d or v_pages.shape != pool:
        raise ValueError(f"{where}: pools must be [num_pages, page, Hkv, {d}], got {tuple(pool)} and "
                         f"{tuple(v_pages.shape)}")
    num_pages, page, Hkv, _ = pool
    maxp = block_table.shape[-1]
    _need(where, torch.bfloat16, dev, True, q, k_pages, v_pages)
    _need(where, torch.int32, dev, True, block_table, seqlens_k)
    _shape(where, "block_table", block_table, B, maxp)
    _shape(where, "seqlens_k", seqlens_k, B)
    out, ld = _mass_out(where, mass, out, B, Hkv, maxp * page, dev, stream)
    if n_splits == 0:
        n_splits = _lib.mala_decode_default_splits(B, Hkv, maxp * page, page)
    o = _empty(q.shape, q.dtype, dev, stream)
    lse = _empty((B, Hq), torch.float32, dev, stream)
    kept = _empty((B * Hq,), torch.int32, dev, stream)
    km = None
    if keep_map:
        km = _empty((B, Hq, maxp), torch.uint8, dev, stream)
        if stream is None:
            km.fill_(255)
        else:
            with _on(stream):
                km.fill_(255)
    ws, ws_bytes, _hold = _scratch(where, workspace,
                                   _lib.mala_decode_mass_workspace_size(B, Hq, d, page, maxp, n_splits), dev, stream)
    rc = _lib.mala_decode_paged_mass(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                                     seqlens_k.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                     None if mass is None else mass.data_ptr(), out.data_ptr(), B, Hq, Hkv, num_pages,
                                     page, maxp, d, scale, tau, decay, ld, n_splits, ws, ws_bytes, kept.data_ptr(),
                                     None if km is None else km.data_ptr(), _raw_stream(stream, dev))
    if rc:
        _check(rc, where)
    return o, lse, kept, km, n_splits, out


def evict_select(mass, seqlens_k, budget: int, n_sink: int = 0, n_recent: int = 0, stream=None):
    """Rows that remain of each cache cut down to `budget` rows: mass [B,Hkv,ld] fp32, seqlens_k [B] int32 ->
    (index [B,Hkv,budget] int32 ascending, -1 past the rows there are; new_seqlens [B]; mass [B,Hkv,budget])."""
    import torch
    where = "mala_evict_select"
    dev = _device(where, mass)
    B, Hkv, ld = mass.shape
    _need(where, torch.float32, dev, True, mass)
    _need(where, torch.int32, dev, True, seqlens_k)
    _shape(where, "seqlens_k", seqlens_k, B)
    if budget < 1:
        raise ValueError(f"{where}: budget must be at least 1, got {budget}")
    index = _empty((B, Hkv, budget), torch.int32, dev, stream)
    new = _empty((B,), torch.int32, dev, stream)
    out = _empty((B, Hkv, budget), torch.float32, dev, stream)
    rc = _lib.mala_evict_select(mass.data_ptr(), seqlens_k.data_ptr(), index.data_ptr(), new.data_ptr(),
                                out.data_ptr(), B, Hkv, ld, budget, n_sink, n_recent, budget, _raw_stream(stream, dev))
    if rc:
        _check(rc, where)
    return index, new, out


def evict_gather(index, new_seqlens, k_pages, v_pages, block_table, out_table, k_out=None, v_out=None, stream=None):
    """Copy the rows that remain (as evict_select leaves them) into the pages of out_table [B,max_out_pages], in
    the same pools or in k_out / v_out -> (k_out, v_out)."""
    import torch
    where = "mala_evict_gather"
    dev = _device(where, index)
    B, Hkv, budget = index.shape
    k_out = k_pages if k_out is None else k_out
    v_out = v_pages if v_out is None else v_out
    _need(where, torch.int32, dev, True, index, new_seqlens, block_table, out_table)
    _need(where, torch.bfloat16, dev, True, k_pages, v_pages, k_out, v_out)
    pool, to = k_pages.shape, k_out.shape
    if len(pool) != 4 or len(to) != 4 or pool[2] != Hkv or pool[1:] != to[1:] or v_pages.shape != pool or \
            v_out.shape != to:
        raise ValueError(f"{where}: pools must be [num_pages, page, {Hkv}, d], got {tuple(pool)}, "
                         f"{tuple(v_pages.shape)}, {tuple(to)} and {tuple(v_out.shape)}")
    _shape(where, "new_seqlens", new_seqlens, B)
    maxp, max_out = block_table.shape[-1], out_table.shape[-1]
    _shape(where, "block_table", block_table, B, maxp)
    _shape(where, "out_table", out_table, B, max_out)
    rc = _lib.mala_evict_gather(k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), index.data_ptr(),
                                new_seqlens.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), out_table.data_ptr(), B,
                                Hkv, budget, pool[0], to[0], pool[1], maxp, max_out, pool[3],
                                _raw_stream(stream, dev))
    if rc:
        _check(rc, where)
    return k_out, v_out


def evict(mass, seqlens_k, budget: int, k_pages, v_pages, block_table, out_table, n_sink: int = 0, n_recent: int = 0,
          k_out=None, v_out=None, stream=None):
    """Cut caches down to `budget` rows by collected weight (evict_select, then evict_gather) -> (index,
    new_seqlens, mass); the smaller caches are the pages of out_table."""
    index, new, out = evict_select(mass, seqlens_k, budget, n_sink, n_recent, stream)
    evict_gather(index, new, k_pages, v_pages, block_table, out_table, k_out, v_out, stream)
    return index, new, out
