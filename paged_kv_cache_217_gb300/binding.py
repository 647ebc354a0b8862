"""Thin ctypes binding of libpaged_kv.so (the C ABI in include/paged_kv.h).

Argument marshalling only: tensor shapes become sizes, tensors become device
pointers, the current torch stream becomes the cudaStream_t. Every step of
the path runs in the library's CUDA kernels; there is no fallback. If the
library has not been built, every call raises ``LibraryNotBuilt``.

PyTorch supplies device memory and streams. The split-K workspace is a torch
allocation the binding keeps per (device, stream) and grows on demand.
"""

import ctypes
import functools
import os
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libpaged_kv.so")

STATUS = {0: "PKV_OK", 1: "PKV_ERR_INVALID_ARG", 2: "PKV_ERR_UNSUPPORTED",
          3: "PKV_ERR_OUT_OF_BLOCKS", 4: "PKV_ERR_CUDA", 5: "PKV_ERR_WORKSPACE"}
PKV_F16, PKV_BF16 = 0, 1
BLOCK_SIZE = 16
NOALLOC_SCRATCH_BYTES = 32 << 20   # PKV_NOALLOC_SCRATCH_BYTES
BALANCED = -2                      # pkv_paged_attention_partition: balanced persistent schedule
SHARED_PREFIX = -5                 # pkv_paged_attention_partition: shared-prefix schedule

DEV_FLAGS = {0x1: "BAD_BLOCK_ID", 0x2: "BAD_CONTEXT_LEN", 0x4: "BAD_SLOT", 0x8: "BAD_PAIR",
             0x10: "WAIT_TIMEOUT", 0x20: "BAD_PLAN", 0x40: "OUT_OF_BLOCKS", 0x80: "BAD_POSITION", 0x100: "BAD_START"}
LATENT_DIM, ROPE_DIM = 512, 64     # a latent cache row: the latent vector, then the shared rotary part


class LibraryNotBuilt(RuntimeError):
    pass


class PagedKVError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        self.status_name = STATUS.get(status, str(status))
        super().__init__(f"{self.status_name}: {message}")


class OutOfBlocks(PagedKVError):
    pass


_lib = None
_lib_lock = threading.Lock()

_c_int, _c_i64, _c_sz, _c_f, _c_p = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float, ctypes.c_void_p
_SIGS = {
    "pkv_version": ([], ctypes.c_char_p),
    "pkv_last_error_string": ([], ctypes.c_char_p),
    "pkv_device_status": ([ctypes.POINTER(ctypes.c_uint32), _c_int], _c_int),
    "pkv_paged_attention_decode": ([_c_p] * 6 + [_c_int] * 6 + [_c_f, _c_int, _c_int, _c_p, _c_sz, _c_p],
                                   _c_int),
    "pkv_paged_attention_decode_noalloc": ([_c_p] * 6 + [_c_int] * 6 + [_c_f, _c_int, _c_int, _c_p], _c_int),
    "pkv_paged_attention_decode_planned": ([_c_p] * 6 + [_c_int] * 6 + [_c_f, _c_int, _c_int, _c_p, _c_sz, _c_p],
                                           _c_int),
    "pkv_paged_attention_plan": ([_c_p, _c_p] + [_c_int] * 6 + [_c_p, _c_sz, _c_p], _c_int),
    "pkv_paged_attention_workspace_size": ([_c_int] * 6, _c_sz),
    "pkv_paged_attention_decode_sliding": ([_c_p] * 6 + [_c_int] * 6 + [_c_f, _c_int, _c_int, _c_int, _c_p, _c_sz,
                                                                       _c_p], _c_int),
    "pkv_paged_attention_sliding_workspace_size": ([_c_int] * 7, _c_sz),
    "pkv_paged_attention_partition": ([_c_int] * 6, _c_int),
    "pkv_reshape_and_cache": ([_c_p] * 5 + [_c_int] * 5 + [_c_p], _c_int),
    "pkv_rotary_and_cache": ([_c_p] * 4 + [_c_i64] * 4 + [_c_p] * 2 + [_c_int] * 3 + [_c_p] * 3 + [_c_int] * 6 + [_c_p],
                             _c_int),
    "pkv_paged_prompt_attention": ([_c_p] * 7 + [_c_int] * 7 + [_c_f] + [_c_int] * 3 + [_c_p, _c_sz, _c_p], _c_int),
    "pkv_prompt_workspace_size": ([_c_int] * 6, _c_sz),
    "pkv_paged_prefix_decode": ([_c_p] * 8 + [_c_int] * 7 + [_c_f, _c_int, _c_p, _c_sz, _c_p], _c_int),
    "pkv_prefix_workspace_size": ([_c_int] * 6, _c_sz),
    "pkv_copy_blocks": ([_c_p] * 3 + [_c_int] * 5 + [_c_p], _c_int),
    "pkv_check_copy_pairs": ([_c_p, _c_int, _c_int], _c_int),
    "pkv_reshape_and_cache_int8": ([_c_p, _c_p, _c_int] + [_c_p] * 5 + [_c_int] * 4 + [_c_p], _c_int),
    "pkv_paged_attention_decode_int8": ([_c_p] * 8 + [_c_int] * 6 + [_c_f, _c_int, _c_int, _c_p, _c_sz, _c_p],
                                        _c_int),
    "pkv_paged_attention_decode_int8_planned": ([_c_p] * 8 + [_c_int] * 6 + [_c_f, _c_int, _c_int, _c_p, _c_sz,
                                                                            _c_p], _c_int),
    "pkv_copy_blocks_int8": ([_c_p] * 5 + [_c_int] * 4 + [_c_p], _c_int),
    "pkv_int4_tile_bytes": ([_c_int], _c_sz),
    "pkv_reshape_and_cache_int4": ([_c_p, _c_p, _c_int, _c_p, _c_p] + [_c_int] * 4 + [_c_p], _c_int),
    "pkv_gather_cache_int4": ([_c_p, _c_p, _c_int, _c_p, _c_p] + [_c_int] * 4 + [_c_p], _c_int),
    "pkv_copy_blocks_int4": ([_c_p, _c_p] + [_c_int] * 4 + [_c_p], _c_int),
    "pkv_paged_attention_decode_int4": ([_c_p] * 5 + [_c_int] * 6 + [_c_f, _c_int, _c_int, _c_p, _c_sz, _c_p], _c_int),
    "pkv_int4_workspace_size": ([_c_int] * 6, _c_sz),
    "pkv_latent_cache_write": ([_c_p, _c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_int, _c_int, _c_p], _c_int),
    "pkv_copy_blocks_latent": ([_c_p, _c_p, _c_int, _c_int, _c_p], _c_int),
    "pkv_paged_latent_decode": ([_c_p] * 5 + [_c_int] * 4 + [_c_f, _c_int, _c_p, _c_sz, _c_p], _c_int),
    "pkv_latent_workspace_size": ([_c_int] * 3, _c_sz),
    "pkv_extend_block_tables": ([_c_p] * 3 + [_c_int] * 2 + [_c_p] * 2 + [_c_int] + [_c_p] * 4 +
                                [_c_int, _c_p, _c_p, _c_p, _c_sz, _c_p], _c_int),
    "pkv_extend_workspace_size": ([_c_int] * 2, _c_sz),
    "pkv_release_sequences": ([_c_p] * 3 + [_c_int] * 2 + [_c_p] * 2 + [_c_int, _c_p, _c_p, _c_sz, _c_p], _c_int),
    "pkv_release_workspace_size": ([_c_int], _c_sz),
    "pkv_selftest_bounded_wait": ([ctypes.c_uint32, _c_p], _c_int),
    "pkv_trace_enabled": ([], _c_int),
    "pkv_set_trace_buffer": ([_c_p, _c_int], _c_int),
    "pkv_trace_stamp": ([_c_p, _c_p], _c_int),
    "pkv_trace_empty_grid": ([_c_int, _c_int, _c_int, _c_p], _c_int),
    "pkv_bm_create": ([_c_int, _c_int, _c_p, ctypes.POINTER(_c_p)], _c_int),
    "pkv_bm_destroy": ([_c_p], None),
    "pkv_bm_add_seq": ([_c_p, _c_i64, _c_i64], _c_int),
    "pkv_bm_fork": ([_c_p, _c_i64, _c_i64], _c_int),
    "pkv_bm_append_slot": ([_c_p, _c_i64, _c_p, _c_p, _c_p], _c_int),
    "pkv_bm_append_slots": ([_c_p, _c_p, _c_int, _c_p, _c_p, _c_p], _c_int),
    "pkv_bm_free_seq": ([_c_p, _c_i64], _c_int),
    "pkv_bm_release_before": ([_c_p, _c_i64, _c_i64, _c_p], _c_int),
    "pkv_bm_beam_reorder": ([_c_p, _c_p, _c_int, _c_p, _c_p, _c_int], _c_int),
    "pkv_bm_add_seq_with_prefix": ([_c_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_p], _c_int),
    "pkv_bm_block_tables": ([_c_p, _c_p, _c_int, _c_int, _c_p, _c_p], _c_int),
    "pkv_bm_refcount": ([_c_p, _c_int, _c_p], _c_int),
    "pkv_bm_seq_len": ([_c_p, _c_i64, _c_p], _c_int),
    "pkv_bm_num_free": ([_c_p], _c_int),
    "pkv_bm_num_seqs": ([_c_p], _c_int),
    "pkv_bm_free_stack": ([_c_p, _c_p, _c_int], _c_int),
}


def lib():
    """The loaded library (loaded on first use)."""
    global _lib
    if _lib is None:
        with _lib_lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise LibraryNotBuilt(
                        f"{LIB_PATH} is missing: build it with `python -m paged_kv_cache_217_gb300.build` "
                        "(nvcc, sm_103a); there is no CPU fallback")
                handle = ctypes.CDLL(LIB_PATH)
                for name, (args, res) in _SIGS.items():
                    fn = getattr(handle, name)
                    fn.argtypes = args
                    fn.restype = res
                _lib = handle
    return _lib


def declared_symbols():
    return sorted(_SIGS)


def _check(status, what):
    if status != 0:
        msg = lib().pkv_last_error_string().decode(errors="replace")
        cls = OutOfBlocks if status == 3 else PagedKVError
        raise cls(status, f"{what}: {msg}")


def version():
    return lib().pkv_version().decode()


# ---------------------------------------------------------------------------
# device calls (torch tensors)
# ---------------------------------------------------------------------------
_dtype_codes = {}


def _dtype_code(t):
    code = _dtype_codes.get(t.dtype)
    if code is None:
        import torch
        _dtype_codes.update({torch.float16: PKV_F16, torch.bfloat16: PKV_BF16})
        if t.dtype not in _dtype_codes:
            raise TypeError(f"unsupported dtype {t.dtype} (fp16 or bf16)")
        code = _dtype_codes[t.dtype]
    return code


def _need_cuda(*tensors):
    index = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != index or index < 0:  # (-1: not on a CUDA device)
            raise ValueError("tensors must be on one device" if t.is_cuda else "tensors must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


_handles = None


def _torch_handles():
    """(current device's index, stream handle of a device index): torch's own where it has them (the stream
    object and the device context of its public calls cost 8 us a launch)."""
    global _handles
    if _handles is None:
        import torch
        _handles = (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                    getattr(torch._C, "_cuda_getCurrentRawStream",
                            lambda index: torch.cuda.current_stream(index).cuda_stream))
    return _handles


def _stream_ptr(device):
    index = device.index
    if index is None:
        import torch
        return torch.cuda.current_stream(device).cuda_stream
    return _torch_handles()[1](index)


def _launch(device, what, fn, *args):
    """Calls a launching entry point with ``device`` current and its current
    torch stream as the trailing cudaStream_t: the library looks up per-device
    state (the status word, the no-alloc scratch) on the current device, which
    must be the device of the tensors and of the stream."""
    index, (current, stream) = device.index, _torch_handles()
    if index is not None and index == current():
        status = fn(*args, stream(index))
        if status:
            _check(status, what)
        return
    import torch
    with torch.cuda.device(device):
        _check(fn(*args, _stream_ptr(device)), what)


_workspaces = {}


def _workspace(device, nbytes):
    import torch
    key = (device.index, torch.cuda.current_stream(device).cuda_stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                   partition_size=0):
    return int(lib().pkv_paged_attention_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                         max_blocks_per_seq, partition_size))


def resolved_partition(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, partition_size=0):
    """Schedule a call runs with: BALANCED (-2), -1 (one pass per sequence and KV
    head) or the split-K partition size in tokens; 0 for invalid arguments."""
    return int(lib().pkv_paged_attention_partition(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                   max_blocks_per_seq, partition_size))


def paged_attention_decode(out, q, k_pool, v_pool, block_tables, context_lens, scale,
                           num_kv_heads=None, partition_size=0, workspace=None, planned=False):
    """out[s, h] = softmax(scale * K_s q[s, h]) V_s over the paged cache (in place in ``out``).

    q, out: [S, Hq, D]; k_pool, v_pool: [num_blocks, Hkv, 16, D]; block_tables:
    int32 [S, max_blocks]; context_lens: int32 [S]. ``workspace`` (uint8 CUDA
    tensor) overrides the binding's own workspace. ``planned`` runs
    pkv_paged_attention_decode_planned, which uses the launch plan that
    paged_attention_plan left in the same workspace.
    """
    import torch
    _need_cuda(out, q, k_pool, v_pool, block_tables, context_lens)
    dt = _dtype_code(q)
    if out.dtype != q.dtype or k_pool.dtype != q.dtype or v_pool.dtype != q.dtype:
        raise TypeError("q, out, k_pool and v_pool must share one dtype")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    S, Hq, D = q.shape
    nb, hkv, bs, d2 = k_pool.shape
    if num_kv_heads is None:
        num_kv_heads = hkv
    if bs != BLOCK_SIZE or d2 != D or hkv != num_kv_heads or v_pool.shape != k_pool.shape:
        raise ValueError("pools must be [num_blocks, num_kv_heads, 16, head_dim]")
    if tuple(out.shape) != (S, Hq, D) or block_tables.dim() != 2 or block_tables.shape[0] != S \
            or tuple(context_lens.shape) != (S,):
        raise ValueError("shape mismatch among out, q, block_tables and context_lens")
    mb = block_tables.shape[1]
    need = workspace_size(S, Hq, num_kv_heads, D, mb, partition_size)
    ws_ptr, ws_bytes = None, 0
    if need:
        ws = workspace if workspace is not None else _workspace(q.device, need)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    fn = lib().pkv_paged_attention_decode_planned if planned else lib().pkv_paged_attention_decode
    _launch(q.device, "paged_attention_decode_planned" if planned else "paged_attention_decode", fn,
            out.data_ptr(), q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), block_tables.data_ptr(),
            context_lens.data_ptr(), S, Hq, num_kv_heads, D, mb, nb, float(scale), dt, int(partition_size),
            ws_ptr, ws_bytes)
    return out


def paged_attention_plan(context_lens, block_tables, num_q_heads, num_kv_heads, head_dim, partition_size=0,
                         workspace=None):
    """The decode step's launch plan (pkv_paged_attention_plan) into ``workspace``
    (default: the binding's own workspace of the current stream, which
    paged_attention_decode(planned=True) then reads; threads that plan on one
    stream pass a workspace each). block_tables: int32 [S, max_blocks] (read by
    the shared-prefix schedule's plan)."""
    import torch
    _need_cuda(context_lens, block_tables)
    if context_lens.dtype != torch.int32 or context_lens.dim() != 1 or block_tables.dtype != torch.int32 \
            or block_tables.dim() != 2 or block_tables.shape[0] != context_lens.shape[0]:
        raise TypeError("context_lens must be int32 [S], block_tables int32 [S, max_blocks]")
    S, mb = block_tables.shape
    need = workspace_size(S, num_q_heads, num_kv_heads, head_dim, mb, partition_size)
    ws_ptr, ws_bytes = None, 0
    if need:
        ws = workspace if workspace is not None else _workspace(context_lens.device, need)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    _launch(context_lens.device, "paged_attention_plan", lib().pkv_paged_attention_plan,
            context_lens.data_ptr(), block_tables.data_ptr(), S, int(num_q_heads), int(num_kv_heads),
            int(head_dim), int(mb), int(partition_size), ws_ptr, ws_bytes)


def sliding_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, sliding_window,
                           partition_size=0):
    return int(lib().pkv_paged_attention_sliding_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                                max_blocks_per_seq, sliding_window, partition_size))


def paged_attention_decode_sliding(out, q, k_pool, v_pool, block_tables, context_lens, scale, sliding_window,
                                   partition_size=0, workspace=None):
    """paged_attention_decode over each sequence's last ``sliding_window`` tokens
    (positions max(0, L - W) .. L-1); table entries before them are never read."""
    import torch
    _need_cuda(out, q, k_pool, v_pool, block_tables, context_lens)
    dt = _dtype_code(q)
    if out.dtype != q.dtype or k_pool.dtype != q.dtype or v_pool.dtype != q.dtype:
        raise TypeError("q, out, k_pool and v_pool must share one dtype")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    S, Hq, D = q.shape
    nb, hkv = k_pool.shape[0], k_pool.shape[1]
    if k_pool.shape[2:] != (BLOCK_SIZE, D) or v_pool.shape != k_pool.shape:
        raise ValueError("pools must be [num_blocks, num_kv_heads, 16, head_dim]")
    if tuple(out.shape) != (S, Hq, D) or block_tables.dim() != 2 or block_tables.shape[0] != S \
            or tuple(context_lens.shape) != (S,):
        raise ValueError("shape mismatch among out, q, block_tables and context_lens")
    mb = block_tables.shape[1]
    need = sliding_workspace_size(S, Hq, hkv, D, mb, int(sliding_window), partition_size)
    ws_ptr, ws_bytes = None, 0
    if need:
        ws = workspace if workspace is not None else _workspace(q.device, need)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    _launch(q.device, "paged_attention_decode_sliding", lib().pkv_paged_attention_decode_sliding,
            out.data_ptr(), q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), block_tables.data_ptr(),
            context_lens.data_ptr(), S, Hq, hkv, D, mb, nb, float(scale), dt, int(sliding_window),
            int(partition_size), ws_ptr, ws_bytes)
    return out


def paged_attention_decode_noalloc(out, q, k_pool, v_pool, block_tables, context_lens, scale,
                                   num_kv_heads=None, partition_size=0):
    """paged_attention_decode for callers that cannot allocate device memory.

    Split-K scratch comes from the library's fixed 32 MiB array instead of a
    workspace; see pkv_paged_attention_decode_noalloc in include/paged_kv.h
    (calls overlapping on the GPU race on that array).
    """
    import torch
    _need_cuda(out, q, k_pool, v_pool, block_tables, context_lens)
    dt = _dtype_code(q)
    if out.dtype != q.dtype or k_pool.dtype != q.dtype or v_pool.dtype != q.dtype:
        raise TypeError("q, out, k_pool and v_pool must share one dtype")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    S, Hq, D = q.shape
    nb, hkv = k_pool.shape[0], k_pool.shape[1]
    if num_kv_heads is None:
        num_kv_heads = hkv
    if k_pool.shape[2:] != (BLOCK_SIZE, D) or v_pool.shape != k_pool.shape or hkv != num_kv_heads:
        raise ValueError("pools must be [num_blocks, num_kv_heads, 16, head_dim]")
    if tuple(out.shape) != (S, Hq, D) or block_tables.dim() != 2 or block_tables.shape[0] != S \
            or tuple(context_lens.shape) != (S,):
        raise ValueError("shape mismatch among out, q, block_tables and context_lens")
    _launch(q.device, "paged_attention_decode_noalloc", lib().pkv_paged_attention_decode_noalloc,
            out.data_ptr(), q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), block_tables.data_ptr(),
            context_lens.data_ptr(), S, Hq, num_kv_heads, D, block_tables.shape[1], nb, float(scale), dt,
            int(partition_size))
    return out


def reshape_and_cache(k, v, k_pool, v_pool, slot_mapping):
    """k_pool[slot // 16, :, slot % 16] = k[t] (and v) for every token t with slot >= 0."""
    import torch
    _need_cuda(k, v, k_pool, v_pool, slot_mapping)
    dt = _dtype_code(k)
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    T, hkv, D = k.shape
    if v.shape != k.shape or k_pool.shape[1:] != (hkv, BLOCK_SIZE, D) or v_pool.shape != k_pool.shape \
            or tuple(slot_mapping.shape) != (T,):
        raise ValueError("k, v: [T, Hkv, D]; pools: [num_blocks, Hkv, 16, D]; slot_mapping: [T]")
    if any(x.dtype != k.dtype for x in (v, k_pool, v_pool)):
        raise TypeError("k, v and pools must share one dtype")
    _launch(k.device, "reshape_and_cache", lib().pkv_reshape_and_cache,
            k.data_ptr(), v.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
            slot_mapping.data_ptr(), T, hkv, D, k_pool.shape[0], dt)


def copy_blocks(k_pool, v_pool, src_dst_pairs):
    """Copy block src to block dst in both pools for every row of src_dst_pairs (int64 [n, 2])."""
    import torch
    _need_cuda(k_pool, v_pool, src_dst_pairs)
    dt = _dtype_code(k_pool)
    if src_dst_pairs.dtype != torch.int64 or src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be int64 [n, 2]")
    nb, hkv, bs, D = k_pool.shape
    _launch(k_pool.device, "copy_blocks", lib().pkv_copy_blocks,
            k_pool.data_ptr(), v_pool.data_ptr(), src_dst_pairs.data_ptr(),
            src_dst_pairs.shape[0], hkv, D, nb, dt)


# ---------------------------------------------------------------------------
# INT8 KV cache: int8 codes [num_blocks, Hkv, 16, D], fp32 scales [num_blocks, Hkv, 16]
# ---------------------------------------------------------------------------
def _check_int8_cache(k_cache, v_cache, k_scale, v_scale):
    import torch
    if k_cache.dtype != torch.int8 or v_cache.dtype != torch.int8:
        raise TypeError("k_cache and v_cache must be int8")
    if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
        raise TypeError("k_scale and v_scale must be float32")
    if k_cache.dim() != 4 or k_cache.shape[2] != BLOCK_SIZE or v_cache.shape != k_cache.shape \
            or tuple(k_scale.shape) != tuple(k_cache.shape[:3]) or v_scale.shape != k_scale.shape:
        raise ValueError("caches must be [num_blocks, Hkv, 16, D] and scales [num_blocks, Hkv, 16]")


def reshape_and_cache_int8(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping):
    """Quantise each new K/V row (s = max|x|/127, c = rint(x/s)) into its slot of the INT8 cache."""
    import torch
    _need_cuda(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping)
    dt = _dtype_code(k)
    _check_int8_cache(k_cache, v_cache, k_scale, v_scale)
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    T, hkv, D = k.shape
    if v.shape != k.shape or v.dtype != k.dtype or k_cache.shape[1:] != (hkv, BLOCK_SIZE, D) \
            or tuple(slot_mapping.shape) != (T,):
        raise ValueError("k, v: [T, Hkv, D]; caches: [num_blocks, Hkv, 16, D]; slot_mapping: [T]")
    _launch(k.device, "reshape_and_cache_int8", lib().pkv_reshape_and_cache_int8,
            k.data_ptr(), v.data_ptr(), dt, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), slot_mapping.data_ptr(), T, hkv, D, k_cache.shape[0])


def paged_attention_decode_int8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                                partition_size=0, workspace=None, planned=False):
    """paged_attention_decode over the INT8 cache (K = c_K * s_K, V = c_V * s_V per row). ``planned``
    runs pkv_paged_attention_decode_int8_planned with the plan paged_attention_plan left in the same
    workspace."""
    import torch
    _need_cuda(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens)
    dt = _dtype_code(q)
    _check_int8_cache(k_cache, v_cache, k_scale, v_scale)
    if out.dtype != q.dtype:
        raise TypeError("q and out must share one dtype")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    S, Hq, D = q.shape
    nb, hkv = k_cache.shape[0], k_cache.shape[1]
    if k_cache.shape[3] != D or tuple(out.shape) != (S, Hq, D) or block_tables.dim() != 2 \
            or block_tables.shape[0] != S or tuple(context_lens.shape) != (S,):
        raise ValueError("shape mismatch among out, q, caches, block_tables and context_lens")
    mb = block_tables.shape[1]
    need = workspace_size(S, Hq, hkv, D, mb, partition_size)
    ws_ptr, ws_bytes = None, 0
    if need:
        ws = workspace if workspace is not None else _workspace(q.device, need)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    fn = lib().pkv_paged_attention_decode_int8_planned if planned else lib().pkv_paged_attention_decode_int8
    _launch(q.device, "paged_attention_decode_int8_planned" if planned else "paged_attention_decode_int8", fn,
            out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), S, Hq, hkv, D, mb, nb,
            float(scale), dt, int(partition_size), ws_ptr, ws_bytes)
    return out


def copy_blocks_int8(k_cache, v_cache, k_scale, v_scale, src_dst_pairs):
    """copy_blocks for the INT8 cache: codes and scales of block src go to block dst."""
    import torch
    _need_cuda(k_cache, v_cache, k_scale, v_scale, src_dst_pairs)
    _check_int8_cache(k_cache, v_cache, k_scale, v_scale)
    if src_dst_pairs.dtype != torch.int64 or src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be int64 [n, 2]")
    nb, hkv, _, D = k_cache.shape
    _launch(k_cache.device, "copy_blocks_int8", lib().pkv_copy_blocks_int8,
            k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), src_dst_pairs.data_ptr(), src_dst_pairs.shape[0],
            hkv, D, nb)


# ---------------------------------------------------------------------------
# 4-bit KV cache: uint8 [num_blocks, Hkv, 18 * D], K and V of a (block, KV head) in one tile
# ---------------------------------------------------------------------------
_scratches = {}


def _scratch(device, nbytes):
    """Workspace of one call, or None. Eager calls of a stream share one, which grows to the largest need (an
    allocation a call costs 4 us of host time), whichever threads make them: the library enqueues a call's
    launches together. A call under capture gets memory of its graph's own, so that
    graphs replayed at once, or beside eager calls, never share one."""
    if not nbytes:
        return None
    import torch
    if device.index != _torch_handles()[0]():
        with torch.cuda.device(device):  # whether the stream is capturing is asked of the current device's
            return _scratch(device, nbytes)
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    key = (device.index, _stream_ptr(device))
    ws = _scratches.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _scratches[key] = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
    return ws


def _call_workspace(t, need, workspace):
    """(tensor to keep, address, bytes) of a call's workspace on t's device: the caller's or the binding's own."""
    if not need:
        return None, None, 0
    if workspace is None:
        workspace = _scratch(t.device, need)
    else:
        _need_cuda(t, workspace)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def int4_tile_bytes(head_dim):
    """Bytes of one (block, KV head) tile of the 4-bit cache (18 * head_dim); 0 for head dims it does not take."""
    return int(lib().pkv_int4_tile_bytes(int(head_dim)))


def _check_int4(k, v, kv_cache, slot_mapping):
    import torch
    _need_cuda(k, v, kv_cache, slot_mapping)
    dt = _dtype_code(k)
    if k.dim() != 3 or v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("k and v must be [T, Hkv, D] of one dtype")
    T, hkv, D = k.shape
    if kv_cache.dtype != torch.uint8 or slot_mapping.dtype != torch.int64:
        raise TypeError("kv_cache must be uint8, slot_mapping int64")
    tiles = kv_cache.shape
    if len(tiles) != 3 or tiles[1] != hkv or tiles[2] != 18 * D or slot_mapping.shape != (T,):
        raise ValueError("kv_cache: [num_blocks, Hkv, 18 * D]; slot_mapping: [T]")
    return dt, T, hkv, D, tiles[0]


def reshape_and_cache_int4(k, v, kv_cache, slot_mapping):
    """Quantise each new K/V row to 4 bits (per 64 head dims: offset min x, scale (max x - min x) / 15 in k's
    dtype) into its slot of the 4-bit cache; slots < 0 are skipped."""
    dt, T, hkv, D, nb = _check_int4(k, v, kv_cache, slot_mapping)
    _launch(k.device, "reshape_and_cache_int4", lib().pkv_reshape_and_cache_int4, k.data_ptr(), v.data_ptr(), dt,
            kv_cache.data_ptr(), slot_mapping.data_ptr(), T, hkv, D, nb)


def gather_cache_int4(k, v, kv_cache, slot_mapping):
    """The rows stored at slot_mapping, read back into k and v [T, Hkv, D] (in place; zeros for slots < 0)."""
    dt, T, hkv, D, nb = _check_int4(k, v, kv_cache, slot_mapping)
    _launch(k.device, "gather_cache_int4", lib().pkv_gather_cache_int4, k.data_ptr(), v.data_ptr(), dt,
            kv_cache.data_ptr(), slot_mapping.data_ptr(), T, hkv, D, nb)


def copy_blocks_int4(kv_cache, src_dst_pairs):
    """copy_blocks for the 4-bit cache; pairs (-1, -1) are padding."""
    import torch
    _need_cuda(kv_cache, src_dst_pairs)
    if kv_cache.dtype != torch.uint8 or kv_cache.dim() != 3 or kv_cache.shape[2] % 18:
        raise ValueError("kv_cache must be uint8 [num_blocks, Hkv, 18 * D]")
    if src_dst_pairs.dtype != torch.int64 or src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be int64 [n, 2]")
    nb, hkv, tile = kv_cache.shape
    _launch(kv_cache.device, "copy_blocks_int4", lib().pkv_copy_blocks_int4, kv_cache.data_ptr(),
            src_dst_pairs.data_ptr(), src_dst_pairs.shape[0], hkv, tile // 18, nb)


@functools.lru_cache(maxsize=1024)
def int4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, sliding_window=0):
    return int(lib().pkv_int4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                                             sliding_window))


def paged_attention_decode_int4(out, q, kv_cache, block_tables, context_lens, scale, sliding_window=0,
                                workspace=None):
    """paged_attention_decode over the 4-bit cache (K and V read as offset + code * scale per 64 head dims).

    q, out: [S, Hq, D] of the dtype the cache was written from; kv_cache: uint8
    [num_blocks, Hkv, 18 * D]. ``sliding_window`` > 0 attends over the last
    tokens only. ``workspace`` (uint8 CUDA tensor of int4_workspace_size bytes)
    overrides the binding's own."""
    import torch
    _need_cuda(out, q, kv_cache, block_tables, context_lens)
    dt = _dtype_code(q)
    if out.dtype != q.dtype:
        raise TypeError("q and out must share one dtype")
    if kv_cache.dtype != torch.uint8:
        raise TypeError("kv_cache must be uint8")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    shape, tiles, table = q.shape, kv_cache.shape, block_tables.shape
    if len(shape) != 3 or len(tiles) != 3 or out.shape != shape or tiles[2] != 18 * shape[2] or len(table) != 2 \
            or table[0] != shape[0] or context_lens.shape != (shape[0],):
        raise ValueError("shape mismatch among out, q, kv_cache, block_tables and context_lens")
    window = max(0, int(sliding_window))
    S, Hq, D = shape
    nb, hkv = tiles[0], tiles[1]
    mb = table[1]
    need = int4_workspace_size(S, Hq, hkv, D, mb, window)
    ws, ws_ptr, ws_bytes = _call_workspace(q, need, workspace)
    _launch(q.device, "paged_attention_decode_int4", lib().pkv_paged_attention_decode_int4, out.data_ptr(),
            q.data_ptr(), kv_cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), S, Hq, hkv, D, mb, nb,
            float(scale), dt, window, ws_ptr, ws_bytes)
    return out


# ---------------------------------------------------------------------------
# rotated cache writes, prompt and cross attention, decode behind a shared prefix
# ---------------------------------------------------------------------------
def rotary_and_cache(q_out, q, k, v, positions, cos_sin, k_pool, v_pool, slot_mapping, interleaved=False):
    """reshape_and_cache with queries and keys rotated by position on the way: q_out[t] = R(positions[t]) q[t],
    k_pool[slot // 16, :, slot % 16] = R(positions[t]) k[t], v as it is.

    q, q_out: [T, Hq, D] (q_out may be q; both None: keys and values only); k, v: [T, Hkv, D]; each may be a
    slice of one projection's output. positions: int32 [T], < 0 for padding tokens, which are left out whole.
    cos_sin: float32 [max_positions, rotary_dim], cosines then sines; pairs of elements lie rotary_dim / 2
    apart, next to each other with ``interleaved``."""
    import torch
    _need_cuda(k_pool, v_pool, positions, cos_sin, slot_mapping)
    dt = _dtype_code(k_pool)
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    rows = (k, v) if q is None else (k, v, q, q_out)
    if any(x.dtype != k_pool.dtype for x in rows) or v_pool.dtype != k_pool.dtype:
        raise TypeError("q, k, v and pools must share one dtype")
    if positions.dtype != torch.int32 or slot_mapping.dtype != torch.int64 or cos_sin.dtype != torch.float32:
        raise TypeError("positions must be int32, slot_mapping int64, cos_sin float32")
    index, pool = k_pool.get_device(), k_pool.shape
    if len(pool) != 4 or pool[2] != BLOCK_SIZE or v_pool.shape != pool or cos_sin.dim() != 2 or k.dim() != 3 \
            or (q is not None and q.dim() != 3):
        raise ValueError("pools must be [num_blocks, num_kv_heads, 16, head_dim], cos_sin [max_positions, rotary_dim]")
    nb, hkv, _, D = pool
    T = k.shape[0]
    hq = 0 if q is None else q.shape[1]
    if k.shape != (T, hkv, D) or v.shape != k.shape or positions.shape != (T,) or slot_mapping.shape != (T,) \
            or (q is not None and (q.shape != (T, hq, D) or q_out.shape != q.shape)):
        raise ValueError("q, q_out: [T, Hq, D]; k, v: [T, Hkv, D]; positions and slot_mapping: [T]")
    strides = []
    for x in rows:
        row, head, one = x.stride()
        if x.get_device() != index:
            raise ValueError("tensors must be on one device")
        if T and (one != 1 or (head != D and x.shape[1] > 1)):
            raise ValueError("the heads of a token must be contiguous")
        strides.append(row if T > 1 else x.shape[1] * D)
    ks, vs, qs, qos = strides if q is not None else (*strides, 0, 0)
    _launch(k_pool.device, "rotary_and_cache", lib().pkv_rotary_and_cache, None if q is None else q_out.data_ptr(),
            None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), qos, qs, ks, vs, positions.data_ptr(),
            cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1], int(bool(interleaved)), k_pool.data_ptr(),
            v_pool.data_ptr(), slot_mapping.data_ptr(), T, hq, hkv, D, nb, dt)


@functools.lru_cache(maxsize=1024)
def prompt_workspace_size(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq):
    return int(lib().pkv_prompt_workspace_size(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim,
                                               max_blocks_per_seq))


@functools.lru_cache(maxsize=1024)
def prefix_workspace_size(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq):
    return int(lib().pkv_prefix_workspace_size(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim,
                                               max_blocks_per_seq))


def _check_prompt(out, q, k_pool, v_pool, block_tables, context_lens, *starts):
    import torch
    _need_cuda(out, q, k_pool, v_pool, block_tables, context_lens, *starts)
    dt = _dtype_code(q)
    if out.dtype != q.dtype or k_pool.dtype != q.dtype or v_pool.dtype != q.dtype:
        raise TypeError("q, out, k_pool and v_pool must share one dtype")
    _need_dtype(torch.int32, "tables, lengths and starts", block_tables, context_lens, *starts)
    shape, pool, table = q.shape, k_pool.shape, block_tables.shape
    if len(pool) != 4 or len(shape) != 3 or pool[2] != BLOCK_SIZE or pool[3] != shape[2] or v_pool.shape != pool:
        raise ValueError("q must be [tokens, Hq, head_dim], pools [num_blocks, num_kv_heads, 16, head_dim]")
    if out.shape != shape or len(table) != 2 or context_lens.shape != (table[0],):
        raise ValueError("shape mismatch among out, q, block_tables and context_lens")
    return dt, shape, pool, table


def paged_prompt_attention(out, q, k_pool, v_pool, block_tables, context_lens, query_starts, scale, causal=True,
                           sliding_window=0, workspace=None):
    """out[t, h] = softmax(scale * K_s q[t, h] + mask) V_s over the paged cache, for several query tokens per
    sequence (in place in ``out``).

    q, out: [T, Hq, D], sequence s's tokens from query_starts[s] to query_starts[s + 1] (int32 [S + 1]).
    ``causal``: they are the last of its context_lens[s] tokens and see those up to themselves, the last
    ``sliding_window`` of them when that is > 0 (prompts, chunks of prompts, drafted tokens). Without, they see
    all context_lens[s] tokens (cross attention to an encoder's states). Queries that see nothing get zeros."""
    dt, (T, Hq, D), (nb, hkv, _, _), (S, mb) = _check_prompt(out, q, k_pool, v_pool, block_tables, context_lens,
                                                            query_starts)
    if query_starts.shape != (S + 1,):
        raise ValueError("query_starts must be [S + 1]")
    ws, ws_ptr, ws_bytes = _call_workspace(q, prompt_workspace_size(T, S, Hq, hkv, D, mb), workspace)
    _launch(q.device, "paged_prompt_attention", lib().pkv_paged_prompt_attention, out.data_ptr(), q.data_ptr(),
            k_pool.data_ptr(), v_pool.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
            query_starts.data_ptr(), T, S, Hq, hkv, D, mb, nb, float(scale), dt, int(bool(causal)),
            min(max(0, int(sliding_window)), 2 ** 31 - 1), ws_ptr, ws_bytes)
    return out


def paged_prefix_decode(out, q, k_pool, v_pool, block_tables, context_lens, group_starts, prefix_blocks, scale,
                        workspace=None):
    """paged_attention_decode of groups of sequences that share their first blocks, each shared prefix computed
    once for its whole group (in place in ``out``).

    Group i: sequences group_starts[i] .. group_starts[i + 1] - 1 (int32 [groups + 1]), whose first
    prefix_blocks[i] (int32 [groups]) blocks are those of the group's first sequence. Sequences outside every
    group are computed by themselves."""
    dt, (T, Hq, D), (nb, hkv, _, _), (S, mb) = _check_prompt(out, q, k_pool, v_pool, block_tables, context_lens,
                                                            group_starts, prefix_blocks)
    n = prefix_blocks.numel()
    if T != S or prefix_blocks.shape != (n,) or group_starts.shape != (n + 1,):
        raise ValueError("q must be [S, Hq, head_dim], group_starts [groups + 1], prefix_blocks [groups]")
    ws, ws_ptr, ws_bytes = _call_workspace(q, prefix_workspace_size(S, n, Hq, hkv, D, mb), workspace)
    _launch(q.device, "paged_prefix_decode", lib().pkv_paged_prefix_decode, out.data_ptr(), q.data_ptr(),
            k_pool.data_ptr(), v_pool.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
            group_starts.data_ptr(), prefix_blocks.data_ptr(), n, S, Hq, hkv, D, mb, nb, float(scale), dt, ws_ptr, ws_bytes)
    return out


# ---------------------------------------------------------------------------
# latent attention: one row [latent 512, rotary 64] per token, cache [num_blocks, 16, 576]
# ---------------------------------------------------------------------------
def _check_latent_cache(cache):
    shape = cache.shape
    if len(shape) != 3 or shape[1] != BLOCK_SIZE or shape[2] != LATENT_DIM + ROPE_DIM:
        raise ValueError("a latent cache is [num_blocks, 16, 576]")


def latent_cache_write(latent, rope, cache, slot_mapping):
    """cache[slot // 16, slot % 16] = [latent[t], rope[t]] for every token t with slot >= 0. latent [T, 512]
    and rope [T, 64] may be slices of one tensor (rows a multiple of 8 elements apart)."""
    import torch
    _need_cuda(cache, slot_mapping)
    dt = _dtype_code(cache)
    _check_latent_cache(cache)
    if latent.dtype != cache.dtype or rope.dtype != cache.dtype:
        raise TypeError("latent, rope and cache must share one dtype")
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    index, slots = cache.get_device(), slot_mapping.shape
    if latent.get_device() != index or rope.get_device() != index or len(slots) != 1:
        raise ValueError("tensors must be on one device, slot_mapping [T]")
    T = slots[0]
    if latent.shape != (T, LATENT_DIM) or rope.shape != (T, ROPE_DIM):
        raise ValueError("latent must be [T, 512] and rope [T, 64]")
    (latent_row, one), (rope_row, rope_one) = latent.stride(), rope.stride()
    if T and (one != 1 or rope_one != 1):
        raise ValueError("rows of latent and rope must be contiguous")
    _launch(cache.device, "latent_cache_write", lib().pkv_latent_cache_write, latent.data_ptr(), rope.data_ptr(),
            latent_row, rope_row, dt, cache.data_ptr(), slot_mapping.data_ptr(), T, cache.shape[0])


def copy_blocks_latent(cache, src_dst_pairs):
    """copy_blocks for a latent cache; pairs (-1, -1) are padding."""
    import torch
    _need_cuda(cache, src_dst_pairs)
    _dtype_code(cache)
    _check_latent_cache(cache)
    if src_dst_pairs.dtype != torch.int64 or src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be int64 [n, 2]")
    _launch(cache.device, "copy_blocks_latent", lib().pkv_copy_blocks_latent, cache.data_ptr(),
            src_dst_pairs.data_ptr(), src_dst_pairs.shape[0], cache.shape[0])


@functools.lru_cache(maxsize=1024)
def latent_workspace_size(num_seqs, num_heads, max_blocks_per_seq):
    return int(lib().pkv_latent_workspace_size(int(num_seqs), int(num_heads), int(max_blocks_per_seq)))


def paged_latent_decode(out, q, cache, block_tables, context_lens, scale, workspace=None):
    """out[s, h] = softmax(scale * R_s q[s, h]) C_s, with R_s the sequence's cache rows (576 elements) and C_s
    their first 512 (latent attention, absorbed form). q: [S, H, 576]; out: [S, H, 512]; cache:
    [num_blocks, 16, 576]."""
    import torch
    _need_cuda(out, q, cache, block_tables, context_lens)
    dt = _dtype_code(q)
    _check_latent_cache(cache)
    if out.dtype != q.dtype or cache.dtype != q.dtype:
        raise TypeError("q, out and cache must share one dtype")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    shape, table = q.shape, block_tables.shape
    if len(shape) != 3 or shape[2] != LATENT_DIM + ROPE_DIM or out.shape != (shape[0], shape[1], LATENT_DIM) \
            or len(table) != 2 or table[0] != shape[0] or context_lens.shape != (shape[0],):
        raise ValueError("q: [S, H, 576]; out: [S, H, 512]; block_tables: [S, max_blocks]; context_lens: [S]")
    S, H, _ = shape
    mb = table[1]
    need = latent_workspace_size(S, H, mb)
    ws, ws_ptr, ws_bytes = _call_workspace(q, need, workspace)
    _launch(q.device, "paged_latent_decode", lib().pkv_paged_latent_decode, out.data_ptr(), q.data_ptr(),
            cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), S, H, mb, cache.shape[0], float(scale),
            dt, ws_ptr, ws_bytes)
    return out


# ---------------------------------------------------------------------------
# block tables and slot maps on the device
# ---------------------------------------------------------------------------
def _need_dtype(dtype, what, *tensors):
    for t in tensors:
        if t.dtype != dtype:
            raise TypeError(f"{what} must be {str(dtype)[6:]}")


def extend_block_tables(block_tables, context_lens, new_tokens, free_stack, free_count, slot_mapping, refcounts=None,
                        cow_pairs=None, info=None, new_lens=None, new_free_count=None, workspace=None):
    """Reserves new_tokens[s] more tokens per sequence on the device: takes blocks from the free stack into
    block_tables, writes every new token's slot (sequence after sequence, then -1) into slot_mapping, and the
    lengths and free count after the call into new_lens and new_free_count (default: in place). With
    ``refcounts`` (int32 [num_blocks]) shared last blocks are replaced and their (src, dst) pairs packed into
    ``cow_pairs`` (int64 [S, 2]). All or nothing; see pkv_extend_block_tables for ``info`` (int32 [4]) and flags."""
    import torch
    new_lens = context_lens if new_lens is None else new_lens
    new_free_count = free_count if new_free_count is None else new_free_count
    _need_cuda(block_tables, context_lens, new_tokens, free_stack, free_count, slot_mapping, new_lens, new_free_count,
               *[t for t in (refcounts, cow_pairs, info) if t is not None])
    _need_dtype(torch.int32, "block_tables, lengths, new_tokens, free_stack and free_count", block_tables, context_lens,
                new_tokens, free_stack, free_count, new_lens, new_free_count)
    _need_dtype(torch.int64, "slot_mapping", slot_mapping)
    if block_tables.dim() != 2 or slot_mapping.dim() != 1 or free_stack.dim() != 1:
        raise ValueError("block_tables: [S, max_blocks]; slot_mapping: [n]; free_stack: [num_blocks]")
    S, mb = block_tables.shape
    if context_lens.shape != (S,) or new_tokens.shape != (S,) or new_lens.shape != (S,):
        raise ValueError("context_lens, new_tokens and new_lens must be [S]")
    if free_count.numel() != 1 or new_free_count.numel() != 1:
        raise ValueError("free_count and new_free_count hold one value")
    if (refcounts is None) != (cow_pairs is None):
        raise ValueError("refcounts and cow_pairs come together")
    if refcounts is not None:
        _need_dtype(torch.int32, "refcounts", refcounts)
        _need_dtype(torch.int64, "cow_pairs", cow_pairs)
        if refcounts.shape != free_stack.shape or cow_pairs.shape != (S, 2):
            raise ValueError("refcounts: [num_blocks]; cow_pairs: [S, 2]")
    if info is not None:
        _need_dtype(torch.int32, "info", info)
        if info.numel() != 4:
            raise ValueError("info holds four values")
    n = slot_mapping.shape[0]
    need = int(lib().pkv_extend_workspace_size(S, n))
    ws, ws_ptr, ws_bytes = _call_workspace(block_tables, need, workspace)
    _launch(block_tables.device, "extend_block_tables", lib().pkv_extend_block_tables, block_tables.data_ptr(),
            context_lens.data_ptr(), new_tokens.data_ptr(), S, mb, free_stack.data_ptr(), free_count.data_ptr(),
            free_stack.shape[0], None if refcounts is None else refcounts.data_ptr(), new_lens.data_ptr(),
            new_free_count.data_ptr(), slot_mapping.data_ptr(), n, None if cow_pairs is None else cow_pairs.data_ptr(),
            None if info is None else info.data_ptr(), ws_ptr, ws_bytes)


def release_sequences(block_tables, context_lens, finished, free_stack, free_count, refcounts=None, workspace=None):
    """Drops every sequence with finished[s] != 0 on the device: tables to -1, lengths to 0, and the blocks that
    nothing holds any more onto the free stack in ascending order."""
    import torch
    _need_cuda(block_tables, context_lens, finished, free_stack, free_count,
               *[t for t in (refcounts,) if t is not None])
    _need_dtype(torch.int32, "block_tables, lengths, finished, free_stack, free_count and refcounts", block_tables,
                context_lens, finished, free_stack, free_count, *([] if refcounts is None else [refcounts]))
    if block_tables.dim() != 2 or free_stack.dim() != 1 or free_count.numel() != 1:
        raise ValueError("block_tables: [S, max_blocks]; free_stack: [num_blocks]; free_count holds one value")
    S, mb = block_tables.shape
    if context_lens.shape != (S,) or finished.shape != (S,):
        raise ValueError("context_lens and finished must be [S]")
    if refcounts is not None and refcounts.shape != free_stack.shape:
        raise ValueError("refcounts must be [num_blocks]")
    nb = free_stack.shape[0]
    ws, ws_ptr, ws_bytes = _call_workspace(block_tables, int(lib().pkv_release_workspace_size(nb)), workspace)
    _launch(block_tables.device, "release_sequences", lib().pkv_release_sequences, block_tables.data_ptr(),
            context_lens.data_ptr(), finished.data_ptr(), S, mb, free_stack.data_ptr(), free_count.data_ptr(), nb,
            None if refcounts is None else refcounts.data_ptr(), ws_ptr, ws_bytes)


def check_copy_pairs(pairs, num_blocks):
    """Host check: ids in range, distinct dst, no dst used as a src. Raises PagedKVError."""
    arr = np.ascontiguousarray(np.asarray(pairs, dtype=np.int64).reshape(-1, 2))
    _check(lib().pkv_check_copy_pairs(arr.ctypes.data, arr.shape[0], int(num_blocks)), "check_copy_pairs")


def device_status(clear=True):
    """Flags raised by the kernels' device-side index checks on the current device."""
    v = ctypes.c_uint32(0)
    _check(lib().pkv_device_status(ctypes.byref(v), 1 if clear else 0), "device_status")
    return int(v.value)


def selftest_bounded_wait(limit_us=2000):
    """Runs the bounded-wait self-test on the current device and stream (a wait
    that must run out and raise PKV_DEV_WAIT_TIMEOUT); read it with device_status()."""
    import torch
    _check(lib().pkv_selftest_bounded_wait(int(limit_us), _stream_ptr(torch.device("cuda", torch.cuda.current_device()))),
           "selftest_bounded_wait")


def trace_enabled():
    """True when the loaded library was built with per-CTA tracing (PKV_TRACE=1)."""
    return bool(lib().pkv_trace_enabled())


def set_trace_buffer(buffer):
    """Per-CTA phase timestamps of the following decode calls go into ``buffer``
    (an int64 CUDA tensor of 8 * records words), or stop with None."""
    if buffer is None:
        _check(lib().pkv_set_trace_buffer(None, 0), "set_trace_buffer")
        return
    _need_cuda(buffer)
    import torch
    if buffer.dtype != torch.int64 or buffer.numel() % 8:
        raise ValueError("the trace buffer is int64 with 8 words a record")
    _check(lib().pkv_set_trace_buffer(buffer.data_ptr(), buffer.numel() // 8), "set_trace_buffer")


def trace_stamp(words, index):
    """Enqueues on the current stream a write of the GPU clock (%globaltimer,
    ns) into ``words[index]`` (an int64 CUDA tensor) when the stream gets there."""
    _need_cuda(words)
    import torch
    if words.dtype != torch.int64 or not 0 <= index < words.numel() or not words.is_contiguous():
        raise ValueError("trace_stamp takes a contiguous int64 tensor and an index into it")
    ptr = words.data_ptr() + 8 * int(index)
    _launch(words.device, "trace_stamp", lib().pkv_trace_stamp, ptr)


def trace_empty_grid(device, ctas, threads, smem_bytes):
    """Enqueues on ``device``'s current stream a kernel of ``ctas`` CTAs x
    ``threads`` threads with ``smem_bytes`` of dynamic shared memory that does
    nothing, launched as the decode kernels are: timed between two events it
    is the fixed cost of a launch of that shape."""
    import torch
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("trace_empty_grid needs a CUDA device")
    _launch(device, "trace_empty_grid", lib().pkv_trace_empty_grid, int(ctas), int(threads), int(smem_bytes))


def describe_device_flags(flags):
    return [name for bit, name in DEV_FLAGS.items() if flags & bit]


# ---------------------------------------------------------------------------
# host block manager
# ---------------------------------------------------------------------------
class BlockManager:
    """Host-side KV block manager (free stack, refcounts, copy-on-write).

    Wraps the library's C++ block manager; see pkv_bm_* in include/paged_kv.h.
    """

    def __init__(self, num_blocks, initial_free_order=None, block_size=BLOCK_SIZE):
        self._h = None
        self.num_blocks = int(num_blocks)
        order = None
        if initial_free_order is not None:
            order = np.ascontiguousarray(np.asarray(initial_free_order, dtype=np.int32))
            if order.shape != (self.num_blocks,):
                raise ValueError("initial_free_order must have num_blocks entries")
        h = ctypes.c_void_p()
        _check(lib().pkv_bm_create(self.num_blocks, int(block_size),
                                   None if order is None else order.ctypes.data, ctypes.byref(h)),
               "bm_create")
        self._h = h

    def close(self):
        if self._h is not None:
            lib().pkv_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_seq(self, seq_id, num_tokens):
        _check(lib().pkv_bm_add_seq(self._h, int(seq_id), int(num_tokens)), "bm_add_seq")

    def fork(self, parent, child):
        _check(lib().pkv_bm_fork(self._h, int(parent), int(child)), "bm_fork")

    def append_slot(self, seq_id):
        slot, src, dst = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(lib().pkv_bm_append_slot(self._h, int(seq_id), ctypes.byref(slot), ctypes.byref(src),
                                        ctypes.byref(dst)), "bm_append_slot")
        return slot.value, src.value, dst.value

    def append_slots(self, seq_ids):
        """One slot per sequence, in order; returns (slots int64 [n], pairs int64 [p, 2])."""
        ids = np.ascontiguousarray(np.asarray(seq_ids, dtype=np.int64))
        n = ids.shape[0]
        slots = np.empty(n, dtype=np.int64)
        pairs = np.empty((max(n, 1), 2), dtype=np.int64)
        np_ = ctypes.c_int()
        _check(lib().pkv_bm_append_slots(self._h, ids.ctypes.data, n, slots.ctypes.data, pairs.ctypes.data,
                                         ctypes.byref(np_)), "bm_append_slots")
        return slots, pairs[:np_.value].copy()

    def free_seq(self, seq_id):
        _check(lib().pkv_bm_free_seq(self._h, int(seq_id)), "bm_free_seq")

    def beam_reorder(self, old_ids, parents, new_ids):
        """Beam step: new beam i continues old beam old_ids[parents[i]]; the old beams are dropped."""
        o = np.ascontiguousarray(np.asarray(old_ids, dtype=np.int64))
        p = np.ascontiguousarray(np.asarray(parents, dtype=np.int32))
        n = np.ascontiguousarray(np.asarray(new_ids, dtype=np.int64))
        _check(lib().pkv_bm_beam_reorder(self._h, o.ctypes.data, o.shape[0], p.ctypes.data, n.ctypes.data,
                                         n.shape[0]), "bm_beam_reorder")

    def add_seq_with_prefix(self, seq_id, num_tokens, donor, prefix_tokens):
        """New sequence sharing the whole blocks of its common prefix with `donor`;
        returns the number of shared positions (a multiple of 16)."""
        out = ctypes.c_int64()
        _check(lib().pkv_bm_add_seq_with_prefix(self._h, int(seq_id), int(num_tokens), int(donor),
                                                int(prefix_tokens), ctypes.byref(out)), "bm_add_seq_with_prefix")
        return out.value

    def release_before(self, seq_id, first_token):
        """Drops the sequence's hold on blocks wholly before position first_token
        (their table entries become -1); returns how many entries were dropped."""
        n = ctypes.c_int()
        _check(lib().pkv_bm_release_before(self._h, int(seq_id), int(first_token), ctypes.byref(n)),
               "bm_release_before")
        return n.value

    def block_tables(self, seq_ids, max_blocks_per_seq):
        ids = np.ascontiguousarray(np.asarray(seq_ids, dtype=np.int64))
        n = ids.shape[0]
        table = np.empty((n, int(max_blocks_per_seq)), dtype=np.int32)
        lens = np.empty(n, dtype=np.int32)
        _check(lib().pkv_bm_block_tables(self._h, ids.ctypes.data, n, int(max_blocks_per_seq),
                                         table.ctypes.data, lens.ctypes.data), "bm_block_tables")
        return table, lens

    def block_table(self, seq_id):
        n = -(-self.seq_len(seq_id) // BLOCK_SIZE)
        t, _ = self.block_tables([seq_id], max(n, 1))
        return t[0, :n].tolist()

    def refcount(self, block):
        out = ctypes.c_int32()
        _check(lib().pkv_bm_refcount(self._h, int(block), ctypes.byref(out)), "bm_refcount")
        return out.value

    def seq_len(self, seq_id):
        out = ctypes.c_int64()
        _check(lib().pkv_bm_seq_len(self._h, int(seq_id), ctypes.byref(out)), "bm_seq_len")
        return out.value

    def num_free(self):
        return int(lib().pkv_bm_num_free(self._h))

    def num_seqs(self):
        return int(lib().pkv_bm_num_seqs(self._h))

    def free_stack(self):
        n = int(lib().pkv_bm_free_stack(self._h, None, 0))
        out = np.empty(max(n, 1), dtype=np.int32)
        lib().pkv_bm_free_stack(self._h, out.ctypes.data, n)
        return out[:n].tolist()
