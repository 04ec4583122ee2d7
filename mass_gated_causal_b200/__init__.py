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
_lib.mala_decode_mass_workspace_size.argtypes = [_i] * 7
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


def mala_decode_mass_workspace_size(B, Hq, Hkv, d, page_size, max_pages_per_seq, n_splits) -> int:
    return int(_lib.mala_decode_mass_workspace_size(B, Hq, Hkv, d, page_size, max_pages_per_seq, n_splits))


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
# Checks of the tensors, allocation and the C call are in mala_torch.so (csrc/mala_torch.cpp): these
# calls are short on the GPU, and Python around ctypes took several times as long.
_native = None


def _load_native():
    global _native
    import importlib.util

    import torch  # noqa: F401  (its libraries, which the module links to)
    path = os.path.join(_HERE, "mala_torch.so")
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing (run `python mass_gated_causal_b200/build.py`)")
    spec = importlib.util.spec_from_file_location("mala_torch", path)
    native = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(native)
    native.set_error_class(MalaError)
    _native = native  # only now, for other threads and after a load that failed
    return native


def _rope_flags(adjacent, cyclic):
    return (MALA_ROPE_ADJACENT if adjacent else 0) | (MALA_ROPE_CYCLIC if cyclic else 0)


def rope(q, k, v, positions, inv_freq, sections=None, adjacent: bool = False, cyclic: bool = False, out=None,
         stream=None):
    """Rotary positions: q [..., Hq, d], k and v [..., Hkv, d] bf16 (strided views of a fused projection's
    output will do; any may be None), positions [n_axes, T] int32 (one axis: [T]; T may be the axes "..."),
    inv_freq [rotary_dim / 2] fp32, sections: pairs per axis (None: one axis) -> contiguous (q, k, v), or
    out = (q, k, v) to write to."""
    return (_native or _load_native()).rope(q, k, v, positions, inv_freq, sections, _rope_flags(adjacent, cyclic), out,
                                            stream)


def rope_backward(dq, dk, dv, positions, inv_freq, sections=None, adjacent: bool = False, cyclic: bool = False,
                  out=None, stream=None):
    """Gradient of rope: dq, dk, dv of its outputs -> those of its inputs (out: views of a fused gradient)."""
    return (_native or _load_native()).rope(dq, dk, dv, positions, inv_freq, sections,
                                            _rope_flags(adjacent, cyclic) | MALA_ROPE_INVERSE, out, stream)


def rope_append(q, k, v, positions, inv_freq, k_pages, v_pages, block_table, seqlens_k, cu_seqlens=None, sections=None,
                adjacent: bool = False, cyclic: bool = False, out=None, stream=None):
    """Rotate a serving step's new tokens q [T, Hq, d], k, v [T, Hkv, d] (strided views will do; q may be None)
    and write k and v into the paged cache; seqlens_k counts the new tokens, cu_seqlens [num_seqs+1] says whose
    they are (None: T / num_seqs each) -> rotated q."""
    return (_native or _load_native()).rope_append(q, k, v, positions, inv_freq, k_pages, v_pages, block_table,
                                                   seqlens_k, cu_seqlens, sections, _rope_flags(adjacent, cyclic), out,
                                                   stream)


def key_mass(q, k, lse, scale: float, window: int = 0, mass=None, decay: float = 1.0, out=None, workspace=None,
             stream=None):
    """The attention weight each key collected: q [B,Lq,Hq,d], k [B,Lk,Hkv,d] bf16 and lse [B,Hq,Lq] of a forward
    or prefill call; window: only the last rows count (0: all); mass [B,Hkv,ld] fp32: what earlier calls
    collected, times decay -> mass [B,Hkv,ld] (ld = Lk unless mass or out says more; out may be mass)."""
    return (_native or _load_native()).key_mass(q, k, lse, scale, window, mass, decay, out, workspace, stream)


def key_mass_varlen(q, k, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int, scale: float,
                    window: int = 0, mass=None, decay: float = 1.0, out=None, workspace=None, stream=None):
    """key_mass of a packed batch: q [total_q,Hq,d], k [total_k,Hkv,d], lse [Hq,total_q] as forward_varlen takes
    and leaves them -> mass [num_seqs,Hkv,ld] (ld = max_seqlen_k unless mass or out says more)."""
    return (_native or _load_native()).key_mass_varlen(q, k, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                                                       max_seqlen_k, scale, window, mass, decay, out, workspace, stream)


def decode_paged_mass(q, k_pages, v_pages, block_table, seqlens_k, scale: float, tau: float, mass=None,
                      decay: float = 1.0, out=None, n_splits: int = 0, keep_map: bool = False, workspace=None,
                      stream=None):
    """decode_paged that also collects each key's weight: mass [B,Hkv,ld] fp32 of earlier calls (None: 0), ld >=
    max_pages * page -> (o, lse, kept_tiles, keep_map|None, n_splits (0 without a gate), mass); out: where the masses
    go (may be mass)."""
    return (_native or _load_native()).decode_paged_mass(q, k_pages, v_pages, block_table, seqlens_k, scale, tau, mass,
                                                         decay, out, n_splits, keep_map, workspace, stream)


def evict_select(mass, seqlens_k, budget: int, n_sink: int = 0, n_recent: int = 0, mass_out=None, stream=None):
    """Rows that remain of each cache cut down to `budget` rows: mass [B,Hkv,ld] fp32, seqlens_k [B] int32 ->
    (index [B,Hkv,budget] int32 ascending, -1 past the rows there are; new_seqlens [B]; mass [B,Hkv,budget], or
    mass_out [B,Hkv,ld'], ld' >= budget, filled with 0 past the rows: as long as the smaller cache's decode needs)."""
    return (_native or _load_native()).evict_select(mass, seqlens_k, budget, n_sink, n_recent, mass_out, stream)


def evict_gather(index, new_seqlens, k_pages, v_pages, block_table, out_table, k_out=None, v_out=None, stream=None):
    """Copy the rows that remain (as evict_select leaves them) into the pages of out_table [B,max_out_pages], in
    the same pools or in k_out / v_out -> (k_out, v_out)."""
    return (_native or _load_native()).evict_gather(index, new_seqlens, k_pages, v_pages, block_table, out_table, k_out,
                                                    v_out, stream)


def evict(mass, seqlens_k, budget: int, k_pages, v_pages, block_table, out_table, n_sink: int = 0, n_recent: int = 0,
          k_out=None, v_out=None, mass_out=None, stream=None):
    """Cut caches down to `budget` rows by collected weight (evict_select, then evict_gather) -> (index,
    new_seqlens, mass); the smaller caches are the pages of out_table."""
    return (_native or _load_native()).evict(mass, seqlens_k, budget, k_pages, v_pages, block_table, out_table, n_sink,
                                             n_recent, k_out, v_out, mass_out, stream)
