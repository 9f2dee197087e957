"""Python binding of libkda, the sm_103a library for the KDA recurrent-state path.

Argument marshalling only: every function below turns torch tensors into
device pointers and sizes and calls the C ABI declared in include/kda.h; all
arithmetic runs in the library's CUDA kernels.  There is no CPU fallback: if
libkda.so is missing the import of the library raises.

Entry points (same names as the C ABI):
  kda_chunk_prefill, kda_recurrent_decode, kda_spec_verify, kda_spec_accept, kda_spec_commit,
  kda_spec_accept_commit, kda_conv_compact, kda_slot_copy, kda_slot_copy_noalloc,
  kda_chunk_prefill_workspace_size, kda_slot_copy_workspace_size,
  kda_latent_append, kda_latent_decode, kda_latent_decode_workspace_size, kda_latent_prefill,
  kda_token_logprobs.
"""
from __future__ import annotations

import ctypes
from pathlib import Path

import torch

__all__ = [
    "KDA_BF16", "KDA_F32", "KDA_GATE_LOG", "KDA_BETA_ACT", "KDA_STATE_BF16", "KDA_STATE_F16",
    "KDA_QK_L2NORM", "KDA_F16", "KDA_LATENT_FULL",
    "KdaError", "lib",
    "kda_chunk_prefill", "kda_recurrent_decode", "kda_spec_verify", "kda_spec_accept",
    "kda_spec_commit", "kda_spec_accept_commit", "kda_conv_compact", "kda_slot_copy",
    "kda_slot_copy_noalloc", "kda_chunk_prefill_workspace_size",
    "kda_slot_copy_workspace_size",
    "kda_status_string", "kda_abi_version", "kda_selftest_bounded_wait", "PoolDesc",
    "ConvDesc", "CommitExtras", "RowsDesc",
    "kda_latent_append", "kda_latent_decode", "kda_latent_decode_workspace_size",
    "kda_latent_prefill", "kda_token_logprobs",
]

KDA_BF16, KDA_F32, KDA_F16 = 0, 1, 2
KDA_GATE_LOG, KDA_BETA_ACT, KDA_PREFILL_RECURRENT = 1, 2, 4
KDA_STATE_BF16, KDA_STATE_F16 = 8, 16
KDA_QK_L2NORM = 32
KDA_LATENT_FULL = 64
KDA_DEV_BAD_SLOT, KDA_DEV_BAD_TRACK, KDA_DEV_BAD_ACCEPT = 1, 2, 4
KDA_DEV_BAD_SEQLEN, KDA_DEV_OVERLAP, KDA_DEV_TIMEOUT = 8, 16, 32
KDA_MAX_POOLS = 16

# absent from torch builds without CUDA, which can do no more with this package than import it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)

LIB_PATH = Path(__file__).resolve().parent / "libkda.so"
_lib = None


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {kda_status_string(status)} (status {status})")
        self.status = status


class PoolDesc(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("slot_stride_bytes", ctypes.c_int64),
                ("slot_bytes", ctypes.c_int64), ("num_slots", ctypes.c_int64)]


class ConvDesc(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("slot_stride_bytes", ctypes.c_int64),
                ("row_bytes", ctypes.c_int64), ("n_rows", ctypes.c_int32),
                ("num_slots", ctypes.c_int32)]


class CommitExtras(ctypes.Structure):
    _fields_ = [("convs", ctypes.POINTER(ConvDesc)), ("conv_slot", ctypes.c_void_p),
                ("seq_len0", ctypes.c_void_p), ("block_slot", ctypes.c_void_p),
                ("block_idx_out", ctypes.c_void_p), ("n_convs", ctypes.c_int32),
                ("conv_keep", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class RowsDesc(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


def lib():
    """The loaded C library with argument types set (raises if not built)."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(there is no fallback path)")
        L = ctypes.CDLL(str(LIB_PATH))
        vp, i32, i64, f32, u32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                      ctypes.c_float, ctypes.c_uint32, ctypes.c_size_t)
        L.kda_chunk_prefill.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, vp, i32, i32, i32, i32,
                                        i32, i32, f32, u32, vp, i64, vp, vp, vp, i32, vp, vp,
                                        ctypes.c_int, vp, sz, vp, vp]
        L.kda_recurrent_decode.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, i32, i32, i32, i32,
                                           f32, u32, vp, i64, vp, vp, ctypes.c_int, vp, vp]
        L.kda_spec_verify.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, i32, i32, vp, i32, i32,
                                      i32, f32, u32, vp, i64, vp, vp, vp, vp, ctypes.c_int, vp, vp]
        L.kda_spec_commit.argtypes = [vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, i32, u32, vp,
                                      vp, ctypes.c_int, vp, vp, vp]
        L.kda_spec_accept.argtypes = [vp, vp, vp, i32, i32, vp, vp, vp, vp]
        L.kda_spec_accept_commit.argtypes = [vp, i64, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                             u32, vp, vp, ctypes.c_int, vp, vp, vp,
                                             ctypes.POINTER(CommitExtras), vp, vp]
        L.kda_conv_compact.argtypes = [ctypes.POINTER(ConvDesc), i32, vp, vp, i32, i32, vp, vp]
        L.kda_selftest_bounded_wait.argtypes = [u32, vp, vp, vp]
        L.kda_slot_copy.argtypes = [ctypes.POINTER(PoolDesc), i32, vp, i32, vp, vp, vp, i32, i32,
                                    vp, sz, vp, vp]
        L.kda_slot_copy_noalloc.argtypes = [ctypes.POINTER(PoolDesc), i32, vp, i32, vp, vp, vp,
                                            i32, i32, vp, vp]
        L.kda_slot_copy_noalloc.restype = ctypes.c_int
        L.kda_chunk_prefill_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.kda_chunk_prefill_workspace_size.restype = sz
        L.kda_slot_copy_workspace_size.argtypes = [i64]
        L.kda_slot_copy_workspace_size.restype = sz
        rows = ctypes.POINTER(RowsDesc)
        L.kda_latent_append.argtypes = [vp, i64, vp, f32, ctypes.c_int, i32, i32, i32, vp, vp, i64,
                                        i32, i64, vp, vp]
        L.kda_latent_decode.argtypes = [rows, rows, ctypes.c_int, i32, i32, vp, i32, i32, i32, f32,
                                        vp, i64, i32, i64, vp, i32, vp, rows, ctypes.c_int, vp, vp,
                                        sz, vp, vp]
        L.kda_selftest_latent_decode_give_up.argtypes = L.kda_latent_decode.argtypes + [i32, i32]
        L.kda_selftest_latent_decode_give_up.restype = ctypes.c_int
        L.kda_latent_decode_workspace_size.argtypes = [i32, i32, i32]
        L.kda_latent_decode_workspace_size.restype = sz
        L.kda_latent_prefill.argtypes = [rows, rows, vp, i64, rows, ctypes.c_int, vp, vp, i32, i32,
                                         i32, i32, i32, i32, i32, f32, u32, rows, ctypes.c_int, vp,
                                         vp, vp]
        L.kda_selftest_latent_prefill_give_up.argtypes = L.kda_latent_prefill.argtypes + [i32, i32]
        L.kda_selftest_latent_prefill_give_up.restype = ctypes.c_int
        L.kda_token_logprobs.argtypes = [vp, i64, ctypes.c_int, i32, i32, vp, vp, vp, i32, vp, vp,
                                         vp, vp]
        L.kda_status_string.argtypes = [ctypes.c_int]
        L.kda_status_string.restype = ctypes.c_char_p
        L.kda_abi_version.restype = i32
        for f in ("kda_chunk_prefill", "kda_recurrent_decode", "kda_spec_verify",
                  "kda_spec_accept", "kda_spec_commit", "kda_spec_accept_commit",
                  "kda_conv_compact", "kda_slot_copy", "kda_selftest_bounded_wait",
                  "kda_latent_append", "kda_latent_decode", "kda_latent_prefill",
                  "kda_token_logprobs"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def kda_status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


def kda_abi_version() -> int:
    return int(lib().kda_abi_version())


# --------------------------------------------------------------------------
# marshalling helpers


def _p(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return int(t)
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("libkda takes contiguous CUDA tensors")
    return t.data_ptr()


def _p_any(t):
    """Device pointer of a CUDA tensor whose layout the caller describes itself."""
    if not t.is_cuda:
        raise ValueError("libkda takes CUDA tensors")
    return t.data_ptr()


def _dt(t) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


def _acts(*ts) -> int:
    """The one activation dtype of the given tensors (bf16 or fp32): the C ABI takes a
    single in_dtype for q, k, v, beta and gate, so a mix is rejected here."""
    dts = {t.dtype for t in ts if t is not None}
    if len(dts) != 1:
        raise ValueError(f"activations must share one dtype, got {sorted(map(str, dts))}")
    return _dt(next(t for t in ts if t is not None))


def _idx(t, name):
    """Device pointer of an int32 index tensor (or None)."""
    if t is not None and isinstance(t, torch.Tensor) and t.dtype != torch.int32:
        raise ValueError(f"{name} must be an int32 tensor, got {t.dtype}")
    return _p(t)


def _f32(t, name):
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be an fp32 tensor, got {t.dtype}")
    return _p(t)


def _stream(stream):
    if stream is None:
        # the raw handle: building a Stream object costs 3 us a call
        return _raw_stream(_current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _state_flag(*states) -> int:
    """The state-type flag bit for the given state tensors (None entries are
    ignored); every one of them must have the same dtype."""
    dts = {t.dtype for t in states if t is not None}
    if len(dts) > 1:
        raise ValueError(f"state tensors of different dtypes: {dts}")
    dt = dts.pop() if dts else torch.float32
    if dt == torch.float32:
        return 0
    if dt == torch.bfloat16:
        return KDA_STATE_BF16
    if dt == torch.float16:
        return KDA_STATE_F16
    raise ValueError(f"unsupported state dtype {dt}")


def _check(status: int, where: str):
    if status != 0:
        raise KdaError(status, where)


# --------------------------------------------------------------------------
# entry points


def kda_chunk_prefill_workspace_size(T_tot, N, H, dk=128, dv=128, chunk=64) -> int:
    return int(lib().kda_chunk_prefill_workspace_size(T_tot, N, H, dk, dv, chunk))


def kda_slot_copy_workspace_size(num_slots) -> int:
    """Workspace bytes of kda_slot_copy for pools whose smallest slot count is num_slots."""
    return int(lib().kda_slot_copy_workspace_size(num_slots))


def kda_chunk_prefill(q, k, v, beta_raw, gate_raw, cu_seqlens, out, *, state_pool=None,
                      init_slot=None, final_slot=None, track_chunk_idx=None, track_state=None,
                      scale=1.0, flags=0, chunk=64, workspace=None, dev_status=None, stream=None):
    """Chunked prefill over packed sequences (see include/kda.h)."""
    T_tot, H, dk = q.shape
    dv = v.shape[2]
    N = cu_seqlens.shape[0] - 1
    M = 0 if track_chunk_idx is None else int(track_chunk_idx.shape[-1])
    P = 0 if state_pool is None else int(state_pool.shape[0])
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    in_dt = _acts(q, k, v, beta_raw, gate_raw)
    st = lib().kda_chunk_prefill(
        _p(q), _p(k), _p(v), _p(beta_raw), _p(gate_raw), in_dt, _idx(cu_seqlens, "cu_seqlens"),
        N, T_tot, H, dk, dv, chunk, float(scale),
        int(flags) | _state_flag(state_pool, track_state), _p(state_pool), P,
        _idx(init_slot, "init_slot"), _idx(final_slot, "final_slot"),
        _idx(track_chunk_idx, "track_chunk_idx"), M, _p(track_state), _p(out), _dt(out),
        _p(workspace), ws_bytes, _idx(dev_status, "dev_status"), _stream(stream))
    _check(st, "kda_chunk_prefill")


def kda_recurrent_decode(q, k, v, beta_raw, gate_raw, state_pool, slot, out, *, scale=1.0,
                         flags=0, dev_status=None, stream=None):
    """One token per request, in place on state_pool[slot] (see include/kda.h)."""
    R, H, dk = q.shape
    dv = v.shape[2]
    in_dt = _acts(q, k, v, beta_raw, gate_raw)
    st = lib().kda_recurrent_decode(
        _p(q), _p(k), _p(v), _p(beta_raw), _p(gate_raw), in_dt, R, H, dk, dv, float(scale),
        int(flags) | _state_flag(state_pool), _p(state_pool), int(state_pool.shape[0]),
        _idx(slot, "slot"), _p(out), _dt(out), _idx(dev_status, "dev_status"), _stream(stream))
    _check(st, "kda_recurrent_decode")


def kda_spec_verify(q, k, v, beta_raw, gate_raw, state_pool, ckpt_slot, rec_u, rec_kg, out, *,
                    K, q_len=None, scale=1.0, flags=0, dev_status=None, stream=None):
    """K speculative positions per request from one checkpoint (see include/kda.h)."""
    RK, H, dk = q.shape
    dv = v.shape[2]
    K = int(K)
    if K < 0 or (K > 0 and RK % K):
        raise ValueError(f"q has {RK} rows, not a multiple of K = {K}")
    R = RK // K if K > 0 else int(ckpt_slot.numel())  # K = 0 launches nothing
    in_dt = _acts(q, k, v, beta_raw, gate_raw)
    if rec_kg.dtype != q.dtype:
        raise ValueError(f"rec_kg holds the activations' dtype {q.dtype}, got {rec_kg.dtype}")
    st = lib().kda_spec_verify(
        _p(q), _p(k), _p(v), _p(beta_raw), _p(gate_raw), in_dt, R, K, _idx(q_len, "q_len"), H,
        dk, dv, float(scale), int(flags) | _state_flag(state_pool), _p(state_pool),
        int(state_pool.shape[0]), _idx(ckpt_slot, "ckpt_slot"), _f32(rec_u, "rec_u"),
        _p(rec_kg), _p(out), _dt(out), _idx(dev_status, "dev_status"), _stream(stream))
    _check(st, "kda_spec_verify")


def kda_spec_accept(tokens, sampled, num_accepted, *, q_len=None, next_token=None,
                    dev_status=None, stream=None):
    """Accepted length per request from draft vs sampled ids (see include/kda.h).

    tokens, sampled: int32 CUDA tensors [R, K]."""
    R, K = tokens.shape
    st = lib().kda_spec_accept(_idx(tokens, "tokens"), _idx(sampled, "sampled"),
                               _idx(q_len, "q_len"), R, K, _idx(num_accepted, "num_accepted"),
                               _idx(next_token, "next_token"), _idx(dev_status, "dev_status"),
                               _stream(stream))
    _check(st, "kda_spec_accept")


def kda_spec_commit(state_pool, ckpt_slot, num_accepted, rec_u, rec_kg, *, K, dst_slot=None,
                    q_len=None, flags=0, plan_out=None, dev_status=None, stream=None):
    """Closed-form rebuild at the accepted length (see include/kda.h)."""
    P, H, dv, dk = state_pool.shape
    R = ckpt_slot.shape[0]
    st = lib().kda_spec_commit(
        _p(state_pool), P, _idx(ckpt_slot, "ckpt_slot"), _idx(dst_slot, "dst_slot"),
        _idx(num_accepted, "num_accepted"), _idx(q_len, "q_len"), R, K, H, dk, dv,
        int(flags) | _state_flag(state_pool), _f32(rec_u, "rec_u"), _p(rec_kg), _dt(rec_kg),
        _idx(plan_out, "plan_out"), _idx(dev_status, "dev_status"), _stream(stream))
    _check(st, "kda_spec_commit")


def _conv_descs(convs):
    n = 0 if convs is None else len(convs)
    descs = (ConvDesc * max(n, 1))()
    for i, t in enumerate(convs or ()):
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError("conv tensors need contiguous rows")
        descs[i] = ConvDesc(_p_any(t), t.stride(0) * t.element_size(),
                            t.shape[2] * t.element_size(), t.shape[1], t.shape[0])
    return descs, n


def kda_spec_accept_commit(state_pool, ckpt_slot, tokens, sampled, rec_u, rec_kg, *,
                           dst_slot=None, q_len=None, flags=0, num_accepted=None,
                           next_token=None, plan_out=None, convs=None, conv_slot=None,
                           conv_keep=0, seq_len0=None, block_size=0, block_slot=None,
                           block_idx_out=None, dev_status=None, stream=None):
    """Accepted lengths from token ids, the closed-form rebuild and, optionally, the
    short-convolution windows and the align-mode boundary states, one launch (see
    include/kda.h).  tokens, sampled: int32 CUDA tensors [R, K]; convs: list of CUDA
    tensors [num_slots, rows, channels]."""
    P, H, dv, dk = state_pool.shape
    R, K = tokens.shape
    descs, n = _conv_descs(convs)
    extras = CommitExtras(descs, _idx(conv_slot, "conv_slot"), _idx(seq_len0, "seq_len0"),
                          _idx(block_slot, "block_slot"), _idx(block_idx_out, "block_idx_out"),
                          n, int(conv_keep), int(block_size), 0)
    st = lib().kda_spec_accept_commit(
        _p(state_pool), P, _idx(ckpt_slot, "ckpt_slot"), _idx(dst_slot, "dst_slot"),
        _idx(tokens, "tokens"), _idx(sampled, "sampled"), _idx(q_len, "q_len"), R, K, H, dk, dv,
        int(flags) | _state_flag(state_pool), _f32(rec_u, "rec_u"), _p(rec_kg), _dt(rec_kg),
        _idx(num_accepted, "num_accepted"), _idx(next_token, "next_token"),
        _idx(plan_out, "plan_out"), ctypes.byref(extras), _idx(dev_status, "dev_status"),
        _stream(stream))
    _check(st, "kda_spec_accept_commit")


def kda_conv_compact(convs, slot, num_accepted, keep, *, dev_status=None, stream=None):
    """Short-convolution window after acceptance on every conv tensor (see include/kda.h).

    convs: list of CUDA tensors [num_slots, rows, channels] (slot = first dimension, a row
    contiguous)."""
    descs, n = _conv_descs(convs)
    R = int(slot.numel())
    st = lib().kda_conv_compact(descs, n, _idx(slot, "slot"), _idx(num_accepted, "num_accepted"),
                                R, int(keep), _idx(dev_status, "dev_status"), _stream(stream))
    _check(st, "kda_conv_compact")


def kda_selftest_bounded_wait(polls, dev_status, cycles=None, stream=None):
    """Diagnostic: the kernels' bounded wait on a barrier nothing arrives on (see
    include/kda.h).  dev_status: int32 CUDA tensor; cycles: int64 CUDA tensor or None."""
    st = lib().kda_selftest_bounded_wait(int(polls), _idx(dev_status, "dev_status"), _p(cycles),
                                         _stream(stream))
    _check(st, "kda_selftest_bounded_wait")


def kda_slot_copy(pools, clear_slots, src_slots, dst_offsets, dst_slots, workspace, *,
                  dev_status=None, stream=None):
    """Clear / copy / fan out slots on every pool in one launch (see include/kda.h).

    pools: list of CUDA tensors [num_slots, ...] (slot = first dimension)."""
    descs, n, sets = _slot_sets(pools, clear_slots, src_slots, dst_offsets, dst_slots)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib().kda_slot_copy(descs, n, *sets, _p(workspace), ws_bytes,
                             _idx(dev_status, "dev_status"), _stream(stream))
    _check(st, "kda_slot_copy")


def kda_slot_copy_noalloc(pools, clear_slots, src_slots, dst_offsets, dst_slots, *,
                          dev_status=None, stream=None):
    """The slot copy with the library's own fixed check scratch instead of a workspace
    (pools of at most KDA_SLOT_COPY_NOALLOC_MAX_SLOTS slots; see include/kda.h)."""
    descs, n, sets = _slot_sets(pools, clear_slots, src_slots, dst_offsets, dst_slots)
    st = lib().kda_slot_copy_noalloc(descs, n, *sets, _idx(dev_status, "dev_status"),
                                     _stream(stream))
    _check(st, "kda_slot_copy_noalloc")


def _slot_sets(pools, clear_slots, src_slots, dst_offsets, dst_slots):
    """Pool descriptors and the (pointer, count) arguments of the slot sets."""
    n = len(pools)
    descs = (PoolDesc * max(n, 1))()
    for i, t in enumerate(pools):
        descs[i] = PoolDesc(_p(t), t.stride(0) * t.element_size(),
                            t[0].numel() * t.element_size(), t.shape[0])
    n_clear = 0 if clear_slots is None else int(clear_slots.numel())
    n_src = 0 if src_slots is None else int(src_slots.numel())
    n_dst = 0 if dst_slots is None else int(dst_slots.numel())
    sets = (_idx(clear_slots, "clear_slots"), n_clear, _idx(src_slots, "src_slots"),
            _idx(dst_offsets, "dst_offsets"), _idx(dst_slots, "dst_slots"), n_src, n_dst)
    return descs, n, sets


# --------------------------------------------------------------------------
# latent attention and token log probabilities
#
# These marshal with one pass over each tensor's properties: a torch attribute costs about 0.1 us,
# and at the smallest sizes the marshalling is most of a call.

_i32, _f32t = torch.int32, torch.float32
_ANY_DT = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32, torch.float16: KDA_F16}


def _dt3(t) -> int:
    """Element type of the latent attention and log-probability calls (bf16, fp16 or fp32)."""
    dt = _ANY_DT.get(t.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return dt


def _arr(t, dtype, name, shape=None):
    """Device pointer of a contiguous CUDA tensor of the given dtype and shape."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be a tensor of {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("libkda takes contiguous CUDA tensors")
    return t.data_ptr()


def _rows(t, name):
    """Descriptor of a CUDA tensor [rows, heads, channels] whose channels are contiguous; rows and
    heads may be strided (a view of a wider tensor)."""
    (n, h, _), (rs, hs, cs) = t.shape, t.stride()
    if cs != 1 and n and h:
        raise ValueError(f"{name} needs contiguous channels")
    if not t.is_cuda:
        raise ValueError("libkda takes CUDA tensors")
    # a dimension of one element is never stepped along: torch may give it any stride
    return RowsDesc(t.data_ptr(), rs if n > 1 else 0, hs if h > 1 else 0)


def _one_dtype(what, *ts):
    """The element type that all of the given tensors have."""
    dt = ts[0].dtype
    for t in ts[1:]:
        if t.dtype is not dt:
            raise ValueError(f"{what} must share one dtype, got {sorted({str(x.dtype) for x in ts})}")
    dt = _ANY_DT.get(dt)
    return _dt3(ts[0]) if dt is None else dt


def _pages(cache, width):
    """(pointer, pages, page size, page stride) of a paged cache [P, page_size, width]."""
    P, page, w = cache.shape
    ps, rs, cs = cache.stride()
    if cs != 1 or rs != w:
        raise ValueError("cache must be [pages, page_size, width] with contiguous pages")
    if w != width:
        raise ValueError(f"cache must have rows of {width} channels, got {w}")
    if not cache.is_cuda:
        raise ValueError("libkda takes CUDA tensors")
    return cache.data_ptr(), P, page, ps if P > 1 else page * w


def kda_latent_append(kv, cache, slot, *, weight=None, eps=1e-6, dev_status=None, stream=None):
    """Latent vectors (normalised when weight is given) and rope keys of new tokens into the
    paged cache (see include/kda.h).  kv: [T, 576], rows may be strided."""
    T, width = kv.shape
    ks, cs = kv.stride()
    if cs != 1 and T:
        raise ValueError("kv needs contiguous rows")
    dt = _one_dtype("kv, cache and weight", kv, cache, cache if weight is None else weight)
    slot_p = _arr(slot, _i32, "slot", (T,))
    base, P, page, stride = _pages(cache, width)
    if not kv.is_cuda:
        raise ValueError("libkda takes CUDA tensors")
    st = (_lib or lib()).kda_latent_append(
        kv.data_ptr(), ks if T > 1 else width,
        None if weight is None else _arr(weight, kv.dtype, "weight", (width - 64,)), eps, dt, T,
        width - 64, 64, slot_p, base, P, page, stride,
        None if dev_status is None else _arr(dev_status, _i32, "dev_status"), _stream(stream))
    if st:
        _check(st, "kda_latent_append")


def kda_latent_decode_workspace_size(R, K, H) -> int:
    return int(lib().kda_latent_decode_workspace_size(R, K, H))


def kda_latent_decode(q_latent, q_rope, cache, block_table, seq_len, out, workspace, *, K=1,
                      q_len=None, scale=1.0, lse=None, dev_status=None, stream=None):
    """Absorbed latent attention of K query positions a request over a paged cache (see
    include/kda.h).  q_latent [R*K, H, 512], q_rope [R*K, H, 64] and out [R*K, H, 512] may be
    strided over rows and heads."""
    shape = q_latent.shape
    RK, H, dl = shape
    rope_shape = q_rope.shape
    dr = rope_shape[2]
    R, max_pages = block_table.shape
    if K < 0 or RK != R * K:
        raise ValueError(f"q_latent has {RK} rows, not {R} requests x K = {K}")
    dt = _one_dtype("queries and cache", q_latent, q_rope, cache)
    if rope_shape != (RK, H, dr):
        raise ValueError(f"q_rope must have shape {(RK, H, dr)}, got {tuple(rope_shape)}")
    if out.shape != shape:
        raise ValueError(f"out must have shape {tuple(shape)}, got {tuple(out.shape)}")
    base, P, page, stride = _pages(cache, dl + dr)
    ql, qr, o = _rows(q_latent, "q_latent"), _rows(q_rope, "q_rope"), _rows(out, "out")
    st = (_lib or lib()).kda_latent_decode(
        ql, qr, dt, R, K, None if q_len is None else _arr(q_len, _i32, "q_len", (R,)), H, dl, dr,
        scale, base, P, page, stride, _arr(block_table, _i32, "block_table"), max_pages,
        _arr(seq_len, _i32, "seq_len", (R,)), o, _dt3(out),
        None if lse is None else _arr(lse, _f32t, "lse", (RK, H)), _p(workspace), workspace.nbytes,
        None if dev_status is None else _arr(dev_status, _i32, "dev_status"), _stream(stream))
    if st:
        _check(st, "kda_latent_decode")


def kda_latent_prefill(q, k_nope, k_rope, v, cu_q, cu_k, out, *, scale=1.0, flags=0, lse=None,
                       dev_status=None, stream=None):
    """Expanded latent attention of packed sequences (see include/kda.h).  q [Tq, H, 192],
    k_nope and v [Tk, H, 128] and out [Tq, H, 128] may be strided over rows and heads;
    k_rope [Tk, 64] over rows."""
    Tq, H, dq = q.shape
    k_shape, v_shape, out_shape = k_nope.shape, v.shape, out.shape
    Tk, _, dn = k_shape
    rope_rows, dr = k_rope.shape
    dv = v_shape[2]
    if dq != dn + dr or k_shape[1] != H or v_shape != (Tk, H, dv) or out_shape != (Tq, H, dv):
        for name, t, shape in (("q", q, (Tq, H, dn + dr)), ("k_nope", k_nope, (Tk, H, dn)),
                               ("v", v, (Tk, H, dv)), ("out", out, (Tq, H, dv))):
            if t.shape != shape:
                raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if rope_rows != Tk:
        raise ValueError(f"k_rope must have {Tk} rows, got {rope_rows}")
    krs, cs = k_rope.stride()
    if cs != 1 and Tk:
        raise ValueError("k_rope needs contiguous rows")
    dt = _one_dtype("queries, keys and values", q, k_nope, k_rope, v)
    qd, kd, vd, od = _rows(q, "q"), _rows(k_nope, "k_nope"), _rows(v, "v"), _rows(out, "out")
    if not k_rope.is_cuda:
        raise ValueError("libkda takes CUDA tensors")
    N = cu_q.shape[0] - 1
    st = (_lib or lib()).kda_latent_prefill(
        qd, kd, k_rope.data_ptr(), krs if Tk > 1 else dr, vd, dt, _arr(cu_q, _i32, "cu_q"),
        _arr(cu_k, _i32, "cu_k", (N + 1,)), N, Tq, Tk, H, dn, dr, dv, scale, flags, od, _dt3(out),
        None if lse is None else _arr(lse, _f32t, "lse", (Tq, H)),
        None if dev_status is None else _arr(dev_status, _i32, "dev_status"), _stream(stream))
    if st:
        _check(st, "kda_latent_prefill")


def kda_token_logprobs(logits, tokens, logprob, *, entropy=None, top_ids=None, top_logprobs=None,
                       dev_status=None, stream=None):
    """Log probability of given tokens, entropy and top alternatives of logits rows (see
    include/kda.h).  logits [R, V] (rows may be strided), tokens [R]; top_ids and top_logprobs
    [R, top]."""
    R, V = logits.shape
    rs, cs = logits.stride()
    if cs != 1 and R and V > 1:
        raise ValueError("logits needs contiguous rows")
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs go together")
    top, ids, tl = 0, None, None
    if top_ids is not None:
        top = top_ids.shape[1]
        ids = _arr(top_ids, _i32, "top_ids", (R, top))
        tl = _arr(top_logprobs, _f32t, "top_logprobs", (R, top))
    if not logits.is_cuda:
        raise ValueError("libkda takes CUDA tensors")
    st = (_lib or lib()).kda_token_logprobs(
        logits.data_ptr(), rs if R > 1 else V, _dt3(logits), R, V,
        _arr(tokens, _i32, "tokens", (R,)), _arr(logprob, _f32t, "logprob", (R,)),
        None if entropy is None else _arr(entropy, _f32t, "entropy", (R,)), top, ids, tl,
        None if dev_status is None else _arr(dev_status, _i32, "dev_status"), _stream(stream))
    if st:
        _check(st, "kda_token_logprobs")
