"""ctypes binding over libgqa_attn.so (include/gqa_attn.h).

The functions named like the C entry points take torch tensors, check that
they are dense (the C ABI cannot see strides), pass ``data_ptr()`` values,
sizes and the CUDA stream handle, and raise ``GqaAttnError`` on a non-zero
status.  The calls of a serving step around the attention, which pass many
small tensors, do this natively (``csrc/torch_call.cpp``).  Every step of the
computation runs in the library's kernels; there is no Python or CPU
implementation behind these names.  If the library has not been built, the
first call raises instead of falling back to anything.
"""

from __future__ import annotations

import contextlib
import ctypes
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgqa_attn.so")

GQA_OK = 0
GQA_ERR_INVALID_ARG = -1
GQA_ERR_UNSUPPORTED = -2
GQA_ERR_NOT_DEVICE_PTR = -3
GQA_ERR_CUDA = -4
GQA_ERR_WORKSPACE = -5
GQA_ERR_SCRATCH_LIMIT = -6

GQA_F32 = 0
GQA_BF16 = 1

GQA_DEV_KVLEN_CLAMPED = 1
GQA_DEV_EMPTY_REQUEST = 2
GQA_DEV_WAIT_TIMEOUT = 4
GQA_DEV_BAD_BLOCK = 8
GQA_DEV_OUT_OF_BLOCKS = 16
GQA_DEV_BAD_SLOT = 32
GQA_DEV_BAD_POSITION = 64
GQA_DEV_BAD_INDEX = 128

EXPORTED = (
    "gqa_attn_decode_workspace_size",
    "gqa_attn_decode",
    "gqa_attn_decode_noalloc",
    "gqa_attn_decode_paged",
    "gqa_attn_decode_shared_prefix_workspace_size",
    "gqa_attn_decode_shared_prefix",
    "gqa_attn_decode_shared_prefix_paged",
    "gqa_attn_step_tables",
    "gqa_attn_decode_tree_workspace_size",
    "gqa_attn_decode_tree",
    "gqa_attn_decode_tree_paged",
    "gqa_attn_tree_tables",
    "gqa_attn_compact_rows",
    "gqa_attn_fork_tables",
    "gqa_attn_copy_blocks",
    "gqa_attn_rope_append",
    "gqa_attn_decode_layers_workspace_size",
    "gqa_attn_decode_layers",
    "gqa_attn_quantize_q4",
    "gqa_attn_decode_q4_residual_workspace_size",
    "gqa_attn_decode_q4_residual",
    "gqa_attn_decode_q4_workspace_size",
    "gqa_attn_decode_q4",
    "gqa_attn_prefill",
    "gqa_attn_prefill_varlen",
    "gqa_attn_status_string",
    "gqa_attn_read_device_status",
    "gqa_attn_clear_device_status",
    "gqa_attn_decode_num_splits",
    "gqa_attn_decode_plan_for",
    "gqa_attn_version",
    "gqa_attn_set_plan_override",
    "gqa_attn_set_prefill_interleave_override",
    "gqa_attn_set_wait_test",
    "gqa_attn_set_pointer_checks",
    "gqa_attn_read_prefill_status",
    "gqa_attn_clear_prefill_status",
)

_lib = None


class GqaAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().gqa_attn_status_string(status).decode()
        super().__init__(f"{where}: {msg} ({status})")


def lib() -> ctypes.CDLL:
    """Loads libgqa_attn.so once; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m gqa_attention_kv_decode_gb300.build` "
            "(there is no CPU or Python fallback)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    L.gqa_attn_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
    L.gqa_attn_decode_workspace_size.restype = sz
    L.gqa_attn_decode.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp]
    L.gqa_attn_decode.restype = i32
    L.gqa_attn_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, vp]
    L.gqa_attn_decode_noalloc.restype = i32
    L.gqa_attn_decode_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                        i32, f32, i32, vp, sz, vp]
    L.gqa_attn_decode_paged.restype = i32
    L.gqa_attn_decode_layers_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    L.gqa_attn_decode_layers_workspace_size.restype = sz
    L.gqa_attn_decode_layers.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32, i32, vp,
                                         sz, vp]
    L.gqa_attn_decode_layers.restype = i32
    i64 = ctypes.c_int64
    L.gqa_attn_decode_shared_prefix_workspace_size.argtypes = [i32] * 6
    L.gqa_attn_decode_shared_prefix_workspace_size.restype = sz
    L.gqa_attn_decode_shared_prefix.argtypes = [vp] * 8 + [i32] * 8 + [f32, i32, vp, sz, vp]
    L.gqa_attn_decode_shared_prefix.restype = i32
    L.gqa_attn_decode_shared_prefix_paged.argtypes = [vp] * 8 + [i32] * 10 + [f32, i32, vp, sz, vp]
    L.gqa_attn_decode_shared_prefix_paged.restype = i32
    L.gqa_attn_step_tables.argtypes = [vp] * 12 + [i32] * 6 + [vp, sz, vp]
    L.gqa_attn_step_tables.restype = i32
    L.gqa_attn_rope_append.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, f32, vp, vp, vp, vp, vp, vp, vp] \
        + [i32] * 12 + [vp, sz, vp]
    L.gqa_attn_rope_append.restype = i32
    L.gqa_attn_decode_tree_workspace_size.argtypes = [i32] * 6
    L.gqa_attn_decode_tree_workspace_size.restype = sz
    L.gqa_attn_decode_tree.argtypes = [vp] * 8 + [i32] * 8 + [f32, i32, vp, sz, vp]
    L.gqa_attn_decode_tree.restype = i32
    L.gqa_attn_decode_tree_paged.argtypes = [vp] * 9 + [i32] * 10 + [f32, i32, vp, sz, vp]
    L.gqa_attn_decode_tree_paged.restype = i32
    L.gqa_attn_tree_tables.argtypes = [vp] * 7 + [i32] * 5 + [vp, sz, vp]
    L.gqa_attn_tree_tables.restype = i32
    L.gqa_attn_compact_rows.argtypes = [vp] * 8 + [i32] * 9 + [vp, sz, vp]
    L.gqa_attn_compact_rows.restype = i32
    L.gqa_attn_fork_tables.argtypes = [vp] * 15 + [i32] * 5 + [vp, sz, vp]
    L.gqa_attn_fork_tables.restype = i32
    L.gqa_attn_copy_blocks.argtypes = [vp] * 5 + [i32] * 7 + [vp, sz, vp]
    L.gqa_attn_copy_blocks.restype = i32
    L.gqa_attn_quantize_q4.argtypes = [vp, i64, vp, vp, vp, i64, i64, i32, i32, i32, i32, vp]
    L.gqa_attn_quantize_q4.restype = i32
    L.gqa_attn_decode_q4_residual_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.gqa_attn_decode_q4_residual_workspace_size.restype = sz
    L.gqa_attn_decode_q4_residual.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                              i32, i32, i32, i32, i32, i32, i32, i32, f32, vp, sz, vp]
    L.gqa_attn_decode_q4_residual.restype = i32
    L.gqa_attn_decode_q4_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.gqa_attn_decode_q4_workspace_size.restype = sz
    L.gqa_attn_decode_q4.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                     i32, i32, i32, i32, i32, i32, i32, f32, vp, sz, vp]
    L.gqa_attn_decode_q4.restype = i32
    L.gqa_attn_prefill.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32, i32, i32, vp]
    L.gqa_attn_prefill.restype = i32
    L.gqa_attn_prefill_varlen.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, i32, vp]
    L.gqa_attn_prefill_varlen.restype = i32
    L.gqa_attn_status_string.argtypes = [i32]
    L.gqa_attn_status_string.restype = ctypes.c_char_p
    L.gqa_attn_read_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
    L.gqa_attn_read_device_status.restype = i32
    L.gqa_attn_clear_device_status.argtypes = [vp, vp]
    L.gqa_attn_clear_device_status.restype = i32
    L.gqa_attn_decode_num_splits.argtypes = [i32, i32, i32, i32, i32, i32]
    L.gqa_attn_decode_num_splits.restype = i32
    i32p = ctypes.POINTER(ctypes.c_int32)
    L.gqa_attn_decode_plan_for.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32p, i32p, i32p]
    L.gqa_attn_decode_plan_for.restype = i32
    L.gqa_attn_version.argtypes = []
    L.gqa_attn_version.restype = i32
    L.gqa_attn_set_plan_override.argtypes = [i32, i32]
    L.gqa_attn_set_plan_override.restype = i32
    L.gqa_attn_set_prefill_interleave_override.argtypes = [i32]
    L.gqa_attn_set_prefill_interleave_override.restype = i32
    L.gqa_attn_set_wait_test.argtypes = [ctypes.c_uint64]
    L.gqa_attn_set_wait_test.restype = i32
    L.gqa_attn_set_pointer_checks.argtypes = [i32]
    L.gqa_attn_set_pointer_checks.restype = i32
    L.gqa_attn_read_prefill_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), vp]
    L.gqa_attn_read_prefill_status.restype = i32
    L.gqa_attn_clear_prefill_status.argtypes = [vp]
    L.gqa_attn_clear_prefill_status.restype = i32
    _lib = L
    return L


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GQA_F32
    if t.dtype == torch.bfloat16:
        return GQA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16")


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libgqa_attn must be contiguous")
    return t.data_ptr()


_call_mod = None


def _call():
    """The native half of this module (csrc/torch_call.cpp): checks the tensors
    of the serving-step calls and passes them on."""
    global _call_mod
    if _call_mod is None:
        lib()  # (raises if nothing has been built)
        again = "build it with `python -m gqa_attention_kv_decode_gb300.build`"
        try:
            from . import _torch_call
        except ImportError as e:
            raise RuntimeError(f"_torch_call is missing, or of another Python or torch: {again} ({e})") from e
        if _torch_call.torch_version != torch.__version__:
            raise RuntimeError(f"_torch_call was built for torch {_torch_call.torch_version}, this is "
                               f"{torch.__version__}: {again}")
        _call_mod = _torch_call
    return _call_mod


def _stream(stream):
    if stream is None:
        # (the handle alone: torch.cuda.current_stream() builds a Stream
        # object around it, 2.9 us of a 16 us call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(rc: int, where: str):
    if rc != GQA_OK:
        raise GqaAttnError(rc, where)


# --- entry points (same names as the C ABI) ----------------------------------

def gqa_attn_decode_workspace_size(B, Hq, Hkv, D, max_kv_len, dtype) -> int:
    return lib().gqa_attn_decode_workspace_size(B, Hq, Hkv, D, max_kv_len, dtype)


def gqa_attn_decode_num_splits(B, Hq, Hkv, D, max_kv_len, dtype) -> int:
    return lib().gqa_attn_decode_num_splits(B, Hq, Hkv, D, max_kv_len, dtype)


GQA_PLAN_DECODE, GQA_PLAN_PAGED, GQA_PLAN_Q4 = 0, 1, 2


def gqa_attn_decode_plan_for(B, Hq, Hkv, D, max_kv_len, dtype, num_sms, variant=GQA_PLAN_DECODE):
    """(n_split, chunk, tile) of a decode plan for a device of num_sms SMs."""
    n_split, chunk, tile = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    rc = lib().gqa_attn_decode_plan_for(B, Hq, Hkv, D, max_kv_len, dtype, variant, num_sms, ctypes.byref(n_split),
                                        ctypes.byref(chunk), ctypes.byref(tile))
    _check(rc, "gqa_attn_decode_plan_for")
    return n_split.value, chunk.value, tile.value


def gqa_attn_set_plan_override(decode_splits=0, prefill_kv_split=0) -> None:
    """Tuning and tests only: force the decode split count and the prefill
    KV-split cluster size (0 = the planner's choice)."""
    _check(lib().gqa_attn_set_plan_override(int(decode_splits), int(prefill_kv_split)),
           "gqa_attn_set_plan_override")


def gqa_attn_set_wait_test(stall_ns=0) -> None:
    """Tests only: later decode and prefill launches take the path of a copy
    that never lands (a wait of stall_ns on a barrier nothing arrives on), so
    they report GQA_DEV_WAIT_TIMEOUT; 0 turns it off."""
    _check(lib().gqa_attn_set_wait_test(int(stall_ns)), "gqa_attn_set_wait_test")


def gqa_attn_set_pointer_checks(on=True) -> bool:
    """Whether this thread's calls look up if their pointers are the current
    device's (the calls of a serving step see that by the tensors).  Returns
    the setting before."""
    before = lib().gqa_attn_set_pointer_checks(int(on))
    if before < 0:
        _check(before, "gqa_attn_set_pointer_checks")
    return bool(before)


def gqa_attn_set_prefill_interleave_override(from_pair=-1) -> None:
    """Tuning and tests only: prefill pairs from index from_pair on run as
    single query tiles whose keys the two softmax warpgroups take in turn
    (0 = every tile; past the last pair = none; negative = the planner)."""
    _check(lib().gqa_attn_set_prefill_interleave_override(int(from_pair)),
           "gqa_attn_set_prefill_interleave_override")


@contextlib.contextmanager
def plan_override(decode_splits=0, prefill_kv_split=0, prefill_interleave_from=-1):
    """``with plan_override(...)``: the overrides for the block, then none."""
    gqa_attn_set_plan_override(decode_splits, prefill_kv_split)
    gqa_attn_set_prefill_interleave_override(prefill_interleave_from)
    try:
        yield
    finally:
        gqa_attn_set_plan_override(0, 0)
        gqa_attn_set_prefill_interleave_override(-1)


def gqa_attn_decode(q, k, v, o, kv_lens, scale, workspace, max_kv_len=None, stream=None):
    """q, o [B,Hq,1,D]; k, v [B,Hkv,S_cap,D]; kv_lens int32 [B] or None."""
    B, Hq, Tq, D = q.shape
    Hkv, S_cap = k.shape[1], k.shape[2]
    if Tq != 1:
        raise ValueError("decode takes one query row per request")
    if max_kv_len is None:
        max_kv_len = S_cap
    rc = lib().gqa_attn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(kv_lens), B, Hq, Hkv, D,
                               S_cap, int(max_kv_len), float(scale), _dtype_code(q),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream))
    _check(rc, "gqa_attn_decode")


def gqa_attn_decode_noalloc(q, k, v, o, kv_lens, scale, max_kv_len=None, stream=None):
    """gqa_attn_decode without a workspace: the library's built-in scratch is
    used (for callers that cannot allocate; calls must not overlap on the GPU)."""
    B, Hq, Tq, D = q.shape
    Hkv, S_cap = k.shape[1], k.shape[2]
    if Tq != 1:
        raise ValueError("decode takes one query row per request")
    if max_kv_len is None:
        max_kv_len = S_cap
    rc = lib().gqa_attn_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(kv_lens), B, Hq, Hkv,
                                       D, S_cap, int(max_kv_len), float(scale), _dtype_code(q),
                                       _stream(stream))
    _check(rc, "gqa_attn_decode_noalloc")


def gqa_attn_decode_paged(q, k_new, v_new, k_pool, v_pool, block_table, kv_lens, o, scale, workspace,
                          max_kv_len, stream=None):
    """q, o [B,Hq,1,D]; k_pool, v_pool [num_blocks,Hkv,block_size,D] (modified
    when k_new, v_new [B,Hkv,1,D] are given: the new token goes to row
    kv_lens[b]-1); block_table int32 [B,max_blocks]; kv_lens int32 [B]."""
    B, Hq, Tq, D = q.shape
    num_blocks, Hkv, block_size = k_pool.shape[0], k_pool.shape[1], k_pool.shape[2]
    if Tq != 1:
        raise ValueError("decode takes one query row per request")
    if block_table.dtype != torch.int32 or kv_lens.dtype != torch.int32:
        raise TypeError("block_table and kv_lens are int32")
    rc = lib().gqa_attn_decode_paged(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool),
                                     _ptr(block_table), _ptr(kv_lens), _ptr(o), B, Hq, Hkv, D,
                                     block_size, num_blocks, block_table.shape[1], int(max_kv_len),
                                     float(scale), _dtype_code(q), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "gqa_attn_decode_paged")


def gqa_attn_decode_shared_prefix_workspace_size(B, Hq, Hkv, D, max_prefix_len, max_kv_len) -> int:
    return lib().gqa_attn_decode_shared_prefix_workspace_size(B, Hq, Hkv, D, max_prefix_len, max_kv_len)


def gqa_attn_decode_shared_prefix(q, k_prefix, v_prefix, prefix_len, k, v, kv_lens, o, scale, workspace,
                                  max_prefix_len=None, max_kv_len=None, stream=None):
    """q, o [B,Hq,1,D]; k_prefix, v_prefix [Hkv,P_cap,D] shared by the batch,
    prefix_len int32 [1] or None; k, v [B,Hkv,S_cap,D] own rows behind them,
    kv_lens int32 [B] or None."""
    rc = (_call_mod or _call()).decode_shared_prefix(
        q, k_prefix, v_prefix, prefix_len, k, v, kv_lens, o, scale, workspace, max_prefix_len, max_kv_len,
        None if stream is None else _stream(stream))
    if rc:
        _check(rc, "gqa_attn_decode_shared_prefix")


def gqa_attn_decode_shared_prefix_paged(q, k_pool, v_pool, prefix_table, prefix_len, block_table, kv_lens, o, scale,
                                        workspace, max_prefix_len, max_kv_len, stream=None):
    """q, o [B,Hq,1,D]; k_pool, v_pool [num_blocks,Hkv,block_size,D]; the shared
    rows' blocks prefix_table int32 [blocks] (prefix_len int32 [1] rows, or
    None: max_prefix_len), the own rows' block_table int32 [B,max_blocks]."""
    rc = (_call_mod or _call()).decode_shared_prefix_paged(
        q, k_pool, v_pool, prefix_table, prefix_len, block_table, kv_lens, o, scale, workspace, max_prefix_len,
        max_kv_len, None if stream is None else _stream(stream))
    if rc:
        _check(rc, "gqa_attn_decode_shared_prefix_paged")


def gqa_attn_step_tables(prior_lens, new_lens, block_table, free_blocks, free_count, kv_lens, q_lens, q_starts,
                         positions, slots, q_slots, free_count_out, block_size, q_rows, workspace, stream=None):
    """One step's tables from the lengths (all int32): block_table [B,max_blocks]
    grown in place from the stack free_blocks [num_blocks] (or both, and the
    counts, None for a dense cache of block_size rows a request); writes
    kv_lens, q_lens [B], q_starts [B+1], positions, slots, q_slots [T]."""
    rc = (_call_mod or _call()).step_tables(
        prior_lens, new_lens, block_table, free_blocks, free_count, kv_lens, q_lens, q_starts, positions, slots,
        q_slots, free_count_out, block_size, q_rows, workspace, None if stream is None else _stream(stream))
    if rc:
        _check(rc, "gqa_attn_step_tables")


def gqa_attn_rope_append(q, k, v, q_weight, k_weight, eps, cos_sin, positions, slots, q_slots, q_out, k_cache,
                         v_cache, adjacent, workspace, stream=None):
    """q [T,Hq,D], k, v [T,Hkv,D] (token strides allowed) normed (q_weight,
    k_weight [D] or None) and rotated (cos_sin fp32 [max_pos,rot_dim] or None)
    into q_out [q_groups,Hq,q_rows,D] rows q_slots (None: row t) and k_cache,
    v_cache [num_blocks,Hkv,block_size,D] rows slots; negative slots: padding."""
    rc = (_call_mod or _call()).rope_append(
        q, k, v, q_weight, k_weight, eps, cos_sin, positions, slots, q_slots, q_out, k_cache, v_cache, adjacent,
        workspace, None if stream is None else _stream(stream))
    if rc:
        _check(rc, "gqa_attn_rope_append")


def gqa_attn_decode_tree_workspace_size(B, Hq, Hkv, D, Tq, max_kv_len) -> int:
    return lib().gqa_attn_decode_tree_workspace_size(B, Hq, Hkv, D, Tq, max_kv_len)


def gqa_attn_decode_tree(q, k, v, tree_mask, q_lens, tree_lens, kv_lens, o, scale, workspace, max_kv_len=None,
                         stream=None):
    """q, o [B,Hq,Tq,D]: the last q_lens[b] rows of request b (int32 [B], None:
    Tq) over k, v [B,Hkv,S_cap,D], kv_lens int32 [B] rows; tree_mask int32
    [B,Tq,words] over the last tree_lens[b] rows (None: q_lens), or None: a chain."""
    rc = (_call_mod or _call()).decode_tree(
        q, k, v, tree_mask, q_lens, tree_lens, kv_lens, o, scale, workspace, max_kv_len,
        None if stream is None else _stream(stream))
    if rc:
        _check(rc, "gqa_attn_decode_tree")


def gqa_attn_decode_tree_paged(q, k_pool, v_pool, block_table, tree_mask, q_lens, tree_lens, kv_lens, o, scale,
                               workspace, max_kv_len=None, stream=None):
    """gqa_attn_decode_tree over pools [num_blocks,Hkv,block_size,D] and a
    block_table int32 [B,max_blocks]."""
    rc = (_call_mod or _call()).decode_tree_paged(
        q, k_pool, v_pool, block_table, tree_mask, q_lens, tree_lens, kv_lens, o, scale, workspace, max_kv_len,
        None if stream is None else _stream(stream))
    if rc:
        _check(rc, "gqa_attn_decode_tree_paged")


def gqa_attn_tree_tables(parents, tree_lens, q_lens, kv_lens, q_starts, tree_mask, positions, workspace, stream=None):
    """parents int32 [B,N] -> tree_mask int32 [B,Tq,ceil(N/32)] of the last
    q_lens[b] (None: all) of tree_lens[b] nodes, and positions [T] from
    q_starts[b] on (or kv_lens, q_starts and positions None)."""
    rc = (_call_mod or _call()).tree_tables(parents, tree_lens, q_lens, kv_lens, q_starts, tree_mask, positions,
                                            workspace, None if stream is None else _stream(stream))
    if rc:
        _check(rc, "gqa_attn_tree_tables")


def gqa_attn_compact_rows(path, n_keep, tree_lens, kv_lens, block_table, k_cache, v_cache, kv_lens_out, workspace,
                          stream=None):
    """The tree's rows path int32 [B,P] (the first n_keep[b]) moved together
    behind the rows before it, in k_cache, v_cache [num_blocks,Hkv,block_size,D]
    or [layers,...]; block_table None: a dense cache."""
    rc = (_call_mod or _call()).compact_rows(path, n_keep, tree_lens, kv_lens, block_table, k_cache, v_cache,
                                             kv_lens_out, workspace, None if stream is None else _stream(stream))
    if rc:
        _check(rc, "gqa_attn_compact_rows")


def gqa_attn_fork_tables(src, keep_lens, held_lens, block_table, shared, free_blocks, free_count, block_table_out,
                         kv_lens_out, shared_out, free_blocks_out, free_count_out, copy_src, copy_dst, copy_rows,
                         block_size, workspace, stream=None):
    """New request b is the first keep_lens[b] rows (None: all) of old request
    src[b] (int32 [B], negative: none): its table, its length, the holders and
    the stack afterwards, and the copy it needs (gqa_attn_copy_blocks)."""
    rc = (_call_mod or _call()).fork_tables(
        src, keep_lens, held_lens, block_table, shared, free_blocks, free_count, block_table_out, kv_lens_out,
        shared_out, free_blocks_out, free_count_out, copy_src, copy_dst, copy_rows, block_size, workspace,
        None if stream is None else _stream(stream))
    if rc:
        _check(rc, "gqa_attn_fork_tables")


def gqa_attn_copy_blocks(src, dst, rows, k_cache, v_cache, workspace, stream=None):
    """Block src[i] -> block dst[i] (int32 [n], src negative: none), the first
    rows[i] rows of each head (None: all), in k_cache, v_cache
    [num_blocks,Hkv,block_size,D] or [layers,...]."""
    rc = (_call_mod or _call()).copy_blocks(src, dst, rows, k_cache, v_cache, workspace,
                                            None if stream is None else _stream(stream))
    if rc:
        _check(rc, "gqa_attn_copy_blocks")


def gqa_attn_quantize_q4(src, codes, scale, bias, dst_row0=0, rows=None, group_size=64, stream=None):
    """src bf16 [B,Hkv,S_src,D]; codes uint8 [B,Hkv,S_cap,D/2]; scale, bias fp16
    [B,Hkv,S_cap,D/64]: rows [0, rows) of src go to rows [dst_row0, dst_row0 + rows)."""
    B, Hkv, S_src, D = src.shape
    if src.dtype != torch.bfloat16 or codes.dtype != torch.uint8:
        raise TypeError("bf16 source, uint8 codes")
    if scale.dtype != torch.float16 or bias.dtype != torch.float16:
        raise TypeError("fp16 scale and bias")
    rows = S_src if rows is None else int(rows)
    rc = lib().gqa_attn_quantize_q4(_ptr(src), S_src, _ptr(codes), _ptr(scale), _ptr(bias), codes.shape[2],
                                    int(dst_row0), B * Hkv, rows, D, int(group_size), _stream(stream))
    _check(rc, "gqa_attn_quantize_q4")


def gqa_attn_decode_layers_workspace_size(n_layers, B, Hq, Hkv, D, max_kv_len, dtype) -> int:
    return lib().gqa_attn_decode_layers_workspace_size(n_layers, B, Hq, Hkv, D, max_kv_len, dtype)


def gqa_attn_decode_layers(q, k, v, o, kv_lens, scale, workspace, max_kv_len=None, stream=None):
    """Layers stacked on a leading axis: q, o [NL,B,Hq,1,D]; k, v [NL,B,Hkv,S_cap,D];
    kv_lens int32 [B] shared by the layers, or None."""
    NL, B, Hq, Tq, D = q.shape
    Hkv, S_cap = k.shape[2], k.shape[3]
    if Tq != 1:
        raise ValueError("decode takes one query row per request")
    if max_kv_len is None:
        max_kv_len = S_cap
    rc = lib().gqa_attn_decode_layers(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(kv_lens), NL, B, Hq, Hkv, D,
                                      S_cap, int(max_kv_len), float(scale), _dtype_code(q), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "gqa_attn_decode_layers")


def gqa_attn_decode_q4_residual_workspace_size(B, Hq, Hkv, D, max_quant) -> int:
    return lib().gqa_attn_decode_q4_residual_workspace_size(B, Hq, Hkv, D, max_quant)


def gqa_attn_decode_q4_residual(q, k_codes, k_scale, k_bias, v_codes, v_scale, v_bias, k_res, v_res,
                                n_quant, kv_lens, o, scale, workspace, max_quant=None, group_size=64,
                                stream=None):
    """4-bit cache rows [0, n_quant[b]) then window rows (bf16 k_res, v_res
    [B,Hkv,R_cap,D]) up to kv_lens[b]; q, o bf16 [B,Hq,1,D]."""
    B, Hq, Tq, D = q.shape
    Hkv, S_cap = k_codes.shape[1], k_codes.shape[2]
    R_cap = k_res.shape[2]
    if q.dtype != torch.bfloat16 or k_res.dtype != torch.bfloat16:
        raise TypeError("bf16 q and window")
    max_quant = S_cap if max_quant is None else int(max_quant)
    rc = lib().gqa_attn_decode_q4_residual(_ptr(q), _ptr(k_codes), _ptr(k_scale), _ptr(k_bias),
                                           _ptr(v_codes), _ptr(v_scale), _ptr(v_bias), _ptr(k_res),
                                           _ptr(v_res), _ptr(n_quant), _ptr(kv_lens), _ptr(o), B, Hq, Hkv,
                                           D, S_cap, R_cap, max_quant, int(group_size), float(scale),
                                           _ptr(workspace), workspace.numel() * workspace.element_size(),
                                           _stream(stream))
    _check(rc, "gqa_attn_decode_q4_residual")


def gqa_attn_decode_q4_workspace_size(B, Hq, Hkv, D, max_kv_len) -> int:
    return lib().gqa_attn_decode_q4_workspace_size(B, Hq, Hkv, D, max_kv_len)


def gqa_attn_decode_q4(q, k_codes, k_scale, k_bias, v_codes, v_scale, v_bias, o, kv_lens, scale,
                       workspace, max_kv_len=None, group_size=64, stream=None):
    """q, o bf16 [B,Hq,1,D]; codes uint8 [B,Hkv,S_cap,D/2]; scale/bias fp16 [B,Hkv,S_cap,D/G]."""
    B, Hq, Tq, D = q.shape
    Hkv, S_cap = k_codes.shape[1], k_codes.shape[2]
    if q.dtype != torch.bfloat16 or o.dtype != torch.bfloat16:
        raise TypeError("q4 decode takes bf16 q and o")
    if max_kv_len is None:
        max_kv_len = S_cap
    rc = lib().gqa_attn_decode_q4(_ptr(q), _ptr(k_codes), _ptr(k_scale), _ptr(k_bias),
                                  _ptr(v_codes), _ptr(v_scale), _ptr(v_bias), _ptr(o),
                                  _ptr(kv_lens), B, Hq, Hkv, D, S_cap, int(max_kv_len),
                                  int(group_size), float(scale), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "gqa_attn_decode_q4")


def gqa_attn_prefill(q, k, v, o, kv_len, scale, causal=True, stream=None):
    """q, o [B,Hq,q_len,D]; k, v [B,Hkv,S_cap,D]; keys 0..kv_len-1 visible."""
    B, Hq, q_len, D = q.shape
    Hkv, S_cap = k.shape[1], k.shape[2]
    rc = lib().gqa_attn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, D, q_len,
                                int(kv_len), S_cap, float(scale), 1 if causal else 0,
                                _dtype_code(q), _stream(stream))
    _check(rc, "gqa_attn_prefill")


def gqa_attn_prefill_varlen(q, k, v, o, q_lens, kv_lens, scale, causal=True, stream=None):
    """q, o [B,Hq,Tq_cap,D]; k, v [B,Hkv,S_cap,D]; q_lens, kv_lens int32 [B]:
    request b's q_lens[b] queries aligned to the end of its kv_lens[b] keys."""
    B, Hq, Tq_cap, D = q.shape
    Hkv, S_cap = k.shape[1], k.shape[2]
    if q_lens.dtype != torch.int32 or kv_lens.dtype != torch.int32:
        raise TypeError("q_lens and kv_lens are int32")
    rc = lib().gqa_attn_prefill_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(q_lens), _ptr(kv_lens), B, Hq,
                                       Hkv, D, Tq_cap, S_cap, float(scale), 1 if causal else 0, _dtype_code(q),
                                       _stream(stream))
    _check(rc, "gqa_attn_prefill_varlen")


def gqa_attn_status_string(status: int) -> str:
    return lib().gqa_attn_status_string(status).decode()


def gqa_attn_read_device_status(workspace, stream=None) -> int:
    out = ctypes.c_uint32(0)
    _check(lib().gqa_attn_read_device_status(_ptr(workspace), ctypes.byref(out), _stream(stream)),
           "gqa_attn_read_device_status")
    return out.value


def gqa_attn_clear_device_status(workspace, stream=None):
    _check(lib().gqa_attn_clear_device_status(_ptr(workspace), _stream(stream)),
           "gqa_attn_clear_device_status")


def gqa_attn_read_prefill_status(stream=None) -> int:
    out = ctypes.c_uint32(0)
    _check(lib().gqa_attn_read_prefill_status(ctypes.byref(out), _stream(stream)),
           "gqa_attn_read_prefill_status")
    return out.value


def gqa_attn_clear_prefill_status(stream=None):
    _check(lib().gqa_attn_clear_prefill_status(_stream(stream)), "gqa_attn_clear_prefill_status")


def gqa_attn_version() -> int:
    return lib().gqa_attn_version()


# --- conveniences: allocate outputs / workspaces with torch, then call -------

def _on(stream):
    """The workspace that a call on `stream` makes for itself belongs to that
    stream: one of the current stream would be cleared, and given to the next
    tensor, in an order that the call's kernels do not follow.  (Outputs belong
    to the current stream, as whatever the caller makes for the call does.)"""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        # (the handles 0 to 2 name default streams, which wait for one another)
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) > 2 else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


@contextlib.contextmanager
def _zeros_like(q, stream):
    """An output of which a call writes some rows, the others zeros: filled on the
    call's stream, whose kernels follow.  Where the call is refused the current
    stream, which the memory goes back to, waits for the fill."""
    o = torch.empty_like(q)
    with _on(stream):
        o.zero_()
    try:
        yield o
    except Exception:
        if stream is not None:
            with _on(stream):
                used = torch.cuda.current_stream()
            torch.cuda.current_stream().wait_stream(used)
        raise


def rope_table(max_pos, rot_dim, base=10000.0, device="cuda") -> torch.Tensor:
    """The cos_sin table of gqa_attn_rope_append, fp32 [max_pos, rot_dim]: the
    angles position * base^(-2 i / rot_dim) and their cosines and sines in 64
    bits (an fp32 angle of a far position is off by whole steps of it),
    rounded once."""
    inv = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def decode_workspace(B, Hq, Hkv, D, max_kv_len, dtype, device="cuda") -> torch.Tensor:
    n = gqa_attn_decode_workspace_size(B, Hq, Hkv, D, max_kv_len, dtype)
    if n == 0:
        raise ValueError("invalid decode shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def decode_shared_prefix_workspace(B, Hq, Hkv, D, max_prefix_len, max_kv_len, device="cuda") -> torch.Tensor:
    n = gqa_attn_decode_shared_prefix_workspace_size(B, Hq, Hkv, D, max_prefix_len, max_kv_len)
    if n == 0:
        raise ValueError("invalid decode shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def decode_tree_workspace(B, Hq, Hkv, D, Tq, max_kv_len, device="cuda") -> torch.Tensor:
    n = gqa_attn_decode_tree_workspace_size(B, Hq, Hkv, D, Tq, max_kv_len)
    if n == 0:
        raise ValueError("invalid decode shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def decode_q4_workspace(B, Hq, Hkv, D, max_kv_len, device="cuda") -> torch.Tensor:
    n = gqa_attn_decode_q4_workspace_size(B, Hq, Hkv, D, max_kv_len)
    if n == 0:
        raise ValueError("invalid decode shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def decode(q, k, v, kv_lens=None, scale=None, max_kv_len=None, workspace=None, stream=None):
    B, Hq, _, D = q.shape
    Hkv, S_cap = k.shape[1], k.shape[2]
    max_kv_len = S_cap if max_kv_len is None else int(max_kv_len)
    if scale is None:
        scale = D ** -0.5
    if workspace is None:
        with _on(stream):
            workspace = decode_workspace(B, Hq, Hkv, D, max_kv_len, _dtype_code(q), q.device)
    o = torch.empty_like(q)
    gqa_attn_decode(q, k, v, o, kv_lens, scale, workspace, max_kv_len, stream)
    return o


def decode_q4_residual(q, k_codes, k_scale, k_bias, v_codes, v_scale, v_bias, k_res, v_res, n_quant,
                       kv_lens, max_quant=None, scale=None, workspace=None, stream=None):
    B, Hq, _, D = q.shape
    Hkv, S_cap = k_codes.shape[1], k_codes.shape[2]
    max_quant = S_cap if max_quant is None else int(max_quant)
    if scale is None:
        scale = D ** -0.5
    if workspace is None:
        with _on(stream):
            n = gqa_attn_decode_q4_residual_workspace_size(B, Hq, Hkv, D, max_quant)
            if n == 0:
                raise ValueError("invalid decode shape")
            workspace = torch.zeros(n, dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    gqa_attn_decode_q4_residual(q, k_codes, k_scale, k_bias, v_codes, v_scale, v_bias, k_res, v_res,
                                n_quant, kv_lens, o, scale, workspace, max_quant, stream=stream)
    return o


def decode_paged(q, k_pool, v_pool, block_table, kv_lens, max_kv_len, k_new=None, v_new=None,
                 scale=None, workspace=None, stream=None):
    B, Hq, _, D = q.shape
    Hkv = k_pool.shape[1]
    if scale is None:
        scale = D ** -0.5
    if workspace is None:
        with _on(stream):
            workspace = decode_workspace(B, Hq, Hkv, D, max_kv_len, _dtype_code(q), q.device)
    o = torch.empty_like(q)
    gqa_attn_decode_paged(q, k_new, v_new, k_pool, v_pool, block_table, kv_lens, o, scale, workspace,
                          max_kv_len, stream)
    return o


def decode_shared_prefix(q, k_prefix, v_prefix, k, v, prefix_len=None, kv_lens=None, scale=None,
                         max_prefix_len=None, max_kv_len=None, workspace=None, stream=None):
    B, Hq, _, D = q.shape
    Hkv = k.shape[1]
    max_prefix_len = k_prefix.shape[1] if max_prefix_len is None else int(max_prefix_len)
    max_kv_len = k.shape[2] if max_kv_len is None else int(max_kv_len)
    if scale is None:
        scale = D ** -0.5
    if workspace is None:
        with _on(stream):
            workspace = decode_shared_prefix_workspace(B, Hq, Hkv, D, max_prefix_len, max_kv_len, q.device)
    o = torch.empty_like(q)
    gqa_attn_decode_shared_prefix(q, k_prefix, v_prefix, prefix_len, k, v, kv_lens, o, scale, workspace,
                                  max_prefix_len, max_kv_len, stream)
    return o


def decode_shared_prefix_paged(q, k_pool, v_pool, prefix_table, block_table, kv_lens, max_prefix_len, max_kv_len,
                               prefix_len=None, scale=None, workspace=None, stream=None):
    B, Hq, _, D = q.shape
    Hkv = k_pool.shape[1]
    if scale is None:
        scale = D ** -0.5
    if workspace is None:
        with _on(stream):
            workspace = decode_shared_prefix_workspace(B, Hq, Hkv, D, max_prefix_len, max_kv_len, q.device)
    o = torch.empty_like(q)
    gqa_attn_decode_shared_prefix_paged(q, k_pool, v_pool, prefix_table, prefix_len, block_table, kv_lens, o, scale,
                                        workspace, max_prefix_len, max_kv_len, stream)
    return o


def decode_tree(q, k, v, kv_lens, tree_mask=None, q_lens=None, tree_lens=None, scale=None, max_kv_len=None,
                workspace=None, stream=None):
    B, Hq, Tq, D = q.shape
    max_kv_len = k.shape[2] if max_kv_len is None else int(max_kv_len)
    if scale is None:
        scale = D ** -0.5
    if workspace is None:
        with _on(stream):
            workspace = decode_tree_workspace(B, Hq, k.shape[1], D, Tq, max_kv_len, q.device)
    with _zeros_like(q, stream) as o:
        gqa_attn_decode_tree(q, k, v, tree_mask, q_lens, tree_lens, kv_lens, o, scale, workspace, max_kv_len, stream)
    return o


def decode_tree_paged(q, k_pool, v_pool, block_table, kv_lens, tree_mask=None, q_lens=None, tree_lens=None, scale=None,
                      max_kv_len=None, workspace=None, stream=None):
    B, Hq, Tq, D = q.shape
    max_kv_len = block_table.shape[1] * k_pool.shape[2] if max_kv_len is None else int(max_kv_len)
    if scale is None:
        scale = D ** -0.5
    if workspace is None:
        with _on(stream):
            workspace = decode_tree_workspace(B, Hq, k_pool.shape[1], D, Tq, max_kv_len, q.device)
    with _zeros_like(q, stream) as o:
        gqa_attn_decode_tree_paged(q, k_pool, v_pool, block_table, tree_mask, q_lens, tree_lens, kv_lens, o, scale,
                                   workspace, max_kv_len, stream)
    return o


def decode_q4(q, k_codes, k_scale, k_bias, v_codes, v_scale, v_bias, kv_lens=None, scale=None,
              max_kv_len=None, workspace=None, stream=None):
    B, Hq, _, D = q.shape
    Hkv, S_cap = k_codes.shape[1], k_codes.shape[2]
    max_kv_len = S_cap if max_kv_len is None else int(max_kv_len)
    if scale is None:
        scale = D ** -0.5
    if workspace is None:
        with _on(stream):
            workspace = decode_q4_workspace(B, Hq, Hkv, D, max_kv_len, q.device)
    o = torch.empty_like(q)
    gqa_attn_decode_q4(q, k_codes, k_scale, k_bias, v_codes, v_scale, v_bias, o, kv_lens, scale,
                       workspace, max_kv_len, stream=stream)
    return o


def prefill(q, k, v, kv_len=None, scale=None, causal=True, stream=None):
    D = q.shape[-1]
    kv_len = k.shape[2] if kv_len is None else int(kv_len)
    if scale is None:
        scale = D ** -0.5
    o = torch.empty_like(q)
    gqa_attn_prefill(q, k, v, o, kv_len, scale, causal, stream)
    return o
