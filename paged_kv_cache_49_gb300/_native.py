"""ctypes binding of libpkv (include/pkv.h): argument marshalling only.

Every operation runs in the library's CUDA kernels or its C++ block manager;
torch is used for device memory, streams and dtype views. Importing this
module fails loudly if libpkv.so has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpkv.so")

PKV_OK = 0
PKV_EINVAL = -1
PKV_ENOMEM = -2
PKV_ERANGE = -3
PKV_ECUDA = -4
PKV_ENOSPC = -5
PKV_EUNSUPPORTED = -6
PKV_ESTATE = -7

DEVERR_BLOCK_ID = 0x1
DEVERR_SLOT = 0x2
DEVERR_CONTEXT = 0x4
DEVERR_TIMEOUT = 0x8
DEVERR_QUERY = 0x10
DEVERR_POSITION = 0x20

BLOCK_TOKENS = 16
HEAD_DIM = 128
MAX_GROUP = 8
MAX_SEQS = 4096
MAX_CTAS = 2048
TREE_MAX_DRAFTS = 64

EXPORTED = [
    "pkv_version", "pkv_status_string", "pkv_last_cuda_error", "pkv_read_device_error",
    "pkv_append", "pkv_block_copy", "pkv_attn_workspace_size", "pkv_attn_workspace_init",
    "pkv_attn_decode", "pkv_attn_default_ctas", "pkv_bm_create", "pkv_bm_destroy",
    "pkv_bm_admit", "pkv_bm_fork", "pkv_bm_prepare_append", "pkv_bm_free",
    "pkv_bm_block_table", "pkv_bm_context_len", "pkv_bm_batch_tables", "pkv_bm_stats",
    "pkv_bm_refcount", "pkv_attn_decode_static", "pkv_decode_step", "pkv_attn_decode_ex", "pkv_append_ex",
    "pkv_block_copy_ex", "pkv_bm_create_ex", "pkv_bm_admit_tokens", "pkv_bm_preempt", "pkv_bm_resume",
    "pkv_bm_newest_running", "pkv_bm_slots", "pkv_step_layout", "pkv_decode_step_host",
    "pkv_attn_cascade_workspace_size", "pkv_cascade_staging_size", "pkv_cascade_plan", "pkv_attn_decode_cascade",
    "pkv_attn_decode_wait_test", "pkv_attn_decode_cuda_cores", "pkv_attn_workspace_fixed_bytes",
    "pkv_attn_launch_ctas", "pkv_attn_prefill", "pkv_attn_prefill_workspace_size", "pkv_attn_tree",
    "pkv_qk_norm_rope_append", "pkv_int4_block_bytes", "pkv_append_int4", "pkv_load_int4", "pkv_block_copy_int4",
    "pkv_attn_decode_int4", "pkv_attn_decode_int4_wait_test", "pkv_attn_int4_workspace_size", "pkv_beam_select",
    "pkv_beam_workspace_size", "pkv_bm_reorder",
]
BLOCK_SIZES = (8, 16, 32, 64)
INT4_GROUP_DIMS = (32, 64, 128)


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = _lib.pkv_status_string(status).decode()
        if status == PKV_ECUDA:
            msg += f" ({_lib.pkv_last_cuda_error().decode()})"
        super().__init__(f"{what}: {msg} [{status}]" if what else f"{msg} [{status}]")


class PoolExhausted(PkvError):
    pass


class ReservationExceeded(PkvError):
    pass


class StatsT(ctypes.Structure):
    _fields_ = [
        ("num_blocks", ctypes.c_int32), ("free_blocks", ctypes.c_int32),
        ("used_blocks", ctypes.c_int32), ("shared_blocks", ctypes.c_int32),
        ("spare_blocks", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
        ("ref_sum", ctypes.c_int64), ("cow_copies", ctypes.c_int64),
        ("cached_blocks", ctypes.c_int32), ("cached_idle_blocks", ctypes.c_int32),
        ("preempted_seqs", ctypes.c_int32), ("available_blocks", ctypes.c_int32),
        ("cache_hits", ctypes.c_int64), ("evictions", ctypes.c_int64),
    ]


class StepLayoutT(ctypes.Structure):
    _fields_ = [(name, ctypes.c_size_t) for name in
                ("q", "k_new", "v_new", "slot_mapping", "block_tables", "context_lens", "src_dst_pairs", "bytes")]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python paged_kv_cache_49_gb300/build.py` "
            "(nvcc for sm_103a); there is no fallback implementation")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    f32 = ctypes.c_float
    sig = {
        "pkv_version": (i32, []),
        "pkv_status_string": (ctypes.c_char_p, [i32]),
        "pkv_last_cuda_error": (ctypes.c_char_p, []),
        "pkv_read_device_error": (i32, [vp, vp, i32, vp]),
        "pkv_append": (i32, [vp, vp, vp, i32, vp, vp, i32, i32, i32, vp, vp]),
        "pkv_block_copy": (i32, [vp, vp, vp, i32, i32, i32, i32, vp, vp]),
        "pkv_append_ex": (i32, [vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, vp, vp]),
        "pkv_block_copy_ex": (i32, [vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]),
        "pkv_attn_decode_ex": (i32, [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp, vp]),
        "pkv_attn_workspace_size": (sz, [i32, i32]),
        "pkv_attn_workspace_init": (i32, [vp, sz, vp]),
        "pkv_attn_workspace_fixed_bytes": (sz, []),
        "pkv_attn_decode": (i32, [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp, vp]),
        "pkv_attn_default_ctas": (i32, [i32]),
        "pkv_attn_launch_ctas": (i32, [i32, i32, i32, i32]),
        "pkv_attn_decode_cuda_cores": (i32, [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp,
                                             vp]),
        "pkv_attn_decode_wait_test": (i32, [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp,
                                            i32, vp]),
        "pkv_attn_decode_static": (i32, [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, f32, vp, vp, vp]),
        "pkv_decode_step": (i32, [vp, vp, vp, i32, vp, i32, vp, vp, i32, vp, vp, i32, vp, i32, i32, i32, i32,
                                  f32, i32, vp, sz, vp, vp, vp]),
        "pkv_bm_create": (vp, [i32, i32, vp]),
        "pkv_bm_destroy": (None, [vp]),
        "pkv_bm_admit": (i32, [vp, i32, i32, i32, i32, vp]),
        "pkv_bm_fork": (i32, [vp, i32, i32, vp]),
        "pkv_bm_prepare_append": (i32, [vp, vp, i32, vp, vp, vp]),
        "pkv_bm_free": (i32, [vp, i32]),
        "pkv_bm_block_table": (i32, [vp, i32, vp, i32, vp]),
        "pkv_bm_context_len": (i32, [vp, i32, vp]),
        "pkv_bm_batch_tables": (i32, [vp, vp, i32, vp, i32, vp]),
        "pkv_bm_stats": (i32, [vp, vp]),
        "pkv_bm_refcount": (i32, [vp, i32]),
        "pkv_bm_create_ex": (vp, [i32, i32, vp, i32, i32, i32]),
        "pkv_bm_admit_tokens": (i32, [vp, vp, i32, i32, vp, vp]),
        "pkv_bm_preempt": (i32, [vp, i32, vp]),
        "pkv_bm_resume": (i32, [vp, i32]),
        "pkv_bm_newest_running": (i32, [vp]),
        "pkv_bm_slots": (i32, [vp, i32, i32, i32, vp]),
        "pkv_step_layout": (i32, [i32, i32, i32, i32, i32, i32, vp]),
        "pkv_attn_cascade_workspace_size": (sz, [i32, i32, i32, i32, vp, vp]),
        "pkv_cascade_staging_size": (sz, [i32, i32, i32, i32, vp, vp]),
        "pkv_cascade_plan": (i32, [i32, i32, i32, i32, vp, vp, vp, vp, sz, vp, sz, vp]),
        "pkv_attn_decode_cascade": (i32, [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, f32, i32, vp, vp, vp, sz,
                                          vp, vp]),
        "pkv_attn_prefill_workspace_size": (sz, []),
        "pkv_attn_prefill": (i32, [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32, vp, sz, vp,
                                   vp]),
        "pkv_attn_tree": (i32, [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32, vp,
                                sz, vp, vp]),
        "pkv_qk_norm_rope_append": (i32, [vp, i64, vp, i64, vp, i64, vp, vp, f32, vp, i32, i32, i32, vp, vp, i32, i32,
                                          i32, i32, vp, vp, vp, vp, i32, i32, vp, vp]),
        "pkv_int4_block_bytes": (sz, [i32, i32, i32]),
        "pkv_attn_int4_workspace_size": (sz, []),
        "pkv_append_int4": (i32, [vp, i64, vp, i64, vp, i32, vp, i32, i32, i32, i32, i32, vp, vp]),
        "pkv_load_int4": (i32, [vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp]),
        "pkv_block_copy_int4": (i32, [vp, vp, i32, i32, i32, i32, i32, i32, vp, vp]),
        "pkv_attn_decode_int4": (i32, [vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp,
                                       vp]),
        "pkv_attn_decode_int4_wait_test": (i32, [vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i32, f32, i32, vp, sz,
                                                 vp, i32, vp]),
        "pkv_beam_workspace_size": (sz, [i32, i32, i32, i32]),
        "pkv_beam_select": (i32, [vp, i64, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp,
                                  sz, vp, vp]),
        "pkv_bm_reorder": (i32, [vp, vp, vp, i32]),
        "pkv_decode_step_host": (i32, [vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp, vp,
                                       vp, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()
lib = _lib


def _check(status: int, what: str) -> None:
    if status == PKV_OK:
        return
    if status == PKV_ENOMEM:
        raise PoolExhausted(status, what)
    if status == PKV_ENOSPC:
        raise ReservationExceeded(status, what)
    raise PkvError(status, what)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype, name: str, cuda: bool = True) -> None:
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ---------------------------------------------------------------------------
# device operations


def new_error_word(device=None) -> torch.Tensor:
    """A zeroed device uint32 error word (held as int32) for append / copy."""
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def read_device_error(word: torch.Tensor, clear: bool = True, stream=None) -> int:
    host = ctypes.c_uint32(0)
    _check(_lib.pkv_read_device_error(_ptr(word), ctypes.byref(host), int(clear), _stream(stream)),
           "pkv_read_device_error")
    return host.value


def append(k, v, slot_mapping, k_cache, v_cache, device_error=None, stream=None) -> None:
    """Write k[i], v[i] ([T, Hkv, D] bf16) into slot slot_mapping[i] (int64)."""
    _need(k, torch.bfloat16, "k")
    _need(v, torch.bfloat16, "v")
    _need(slot_mapping, torch.int64, "slot_mapping")
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(v_cache, torch.bfloat16, "v_cache")
    nb, hkv, bt, d = k_cache.shape
    if v_cache.shape != k_cache.shape or bt not in BLOCK_SIZES:
        raise ValueError("caches must be [num_blocks, Hkv, block_tokens in (8, 16, 32, 64), D] and alike")
    T = slot_mapping.numel()
    if k.shape != (T, hkv, d) or v.shape != (T, hkv, d):
        raise ValueError("k, v must be [T, Hkv, D] matching the cache and slot_mapping")
    if bt == BLOCK_TOKENS:
        st = _lib.pkv_append(_ptr(k), _ptr(v), _ptr(slot_mapping), T, _ptr(k_cache), _ptr(v_cache),
                             nb, hkv, d, _ptr(device_error), _stream(stream))
    else:
        st = _lib.pkv_append_ex(_ptr(k), _ptr(v), _ptr(slot_mapping), T, _ptr(k_cache), _ptr(v_cache),
                                nb, hkv, d, bt, _ptr(device_error), _stream(stream))
    _check(st, "pkv_append")


def block_copy(k_cache, v_cache, pairs, device_error=None, stream=None) -> None:
    """Copy physical block pairs[i, 0] onto pairs[i, 1] in both caches."""
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(v_cache, torch.bfloat16, "v_cache")
    _need(pairs, torch.int32, "pairs")
    nb, hkv, bt, d = k_cache.shape
    n = pairs.shape[0] if pairs.numel() else 0
    if n and pairs.shape != (n, 2):
        raise ValueError("pairs must be [n, 2]")
    if bt == BLOCK_TOKENS:
        st = _lib.pkv_block_copy(_ptr(k_cache), _ptr(v_cache), _ptr(pairs) if n else None, n, nb, hkv, d,
                                 _ptr(device_error), _stream(stream))
    else:
        st = _lib.pkv_block_copy_ex(_ptr(k_cache), _ptr(v_cache), _ptr(pairs) if n else None, n, nb, hkv, d, bt,
                                    _ptr(device_error), _stream(stream))
    _check(st, "pkv_block_copy")


def default_ctas(num_seqs: int) -> int:
    return int(_lib.pkv_attn_default_ctas(num_seqs))


def launch_ctas(num_seqs: int, num_kv_heads: int, max_blocks_per_seq: int, block_tokens: int = BLOCK_TOKENS) -> int:
    """CTAs attn_decode launches with num_ctas = 0 for this batch shape."""
    return int(_lib.pkv_attn_launch_ctas(num_seqs, num_kv_heads, max_blocks_per_seq, block_tokens))


class AttentionWorkspace:
    """Device scratch for attn_decode: error word, merge counters and per-CTA
    partials, zeroed once at creation. One workspace serves calls of any
    batch and grid whose partial slots fit in it. attn_decode_int4 leaves more
    partial results a CTA, behind the same counters: with int4 the workspace has
    room for them from the start, else its first such call moves it to a larger
    buffer (not while a graph is captured: fewer CTAs do the work then, as in a
    workspace of fewer bytes)."""

    def __init__(self, num_seqs: int, num_kv_heads: int, device=None, stream=None, int4: bool = False):
        nbytes = int(_lib.pkv_attn_workspace_size(num_seqs, num_kv_heads))
        if nbytes == 0:
            raise PkvError(PKV_EINVAL, "pkv_attn_workspace_size")
        self.num_seqs, self.num_kv_heads, self.nbytes = num_seqs, num_kv_heads, nbytes
        self.int4_nbytes = 0  # of the buffer, where it has room for attn_decode_int4's results
        self._before: list[torch.Tensor] = []  # buffers that captured graphs may still use
        device = torch.device(device or "cuda")
        if int4:
            with torch.cuda.device(device):
                self.int4_nbytes = max(nbytes, int(_lib.pkv_attn_int4_workspace_size()))
        self._take(self.int4_nbytes or nbytes, device, _stream(stream))

    def _take(self, nbytes: int, device, stream: int) -> None:
        self.buffer = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
        off = (-self.buffer.data_ptr()) % 256
        self.tensor = self.buffer[off : off + self.nbytes]
        _check(_lib.pkv_attn_workspace_init(self.tensor.data_ptr(), self.nbytes, stream), "pkv_attn_workspace_init")

    def for_int4(self, stream: int) -> int:
        """Bytes of the workspace for a call of attn_decode_int4 on the current device
        and stream."""
        if not self.int4_nbytes and not torch.cuda.is_current_stream_capturing():
            self._before.append(self.tensor)
            self.int4_nbytes = max(self.nbytes, int(_lib.pkv_attn_int4_workspace_size()))
            self._take(self.int4_nbytes, self.tensor.device, stream)
        return self.int4_nbytes or self.nbytes

    @property
    def ptr(self) -> int:
        return self.tensor.data_ptr()

    @staticmethod
    def fixed_bytes() -> int:
        """Leading bytes that must hold zeros between calls (error word,
        merge counters); the rest is scratch."""
        return int(_lib.pkv_attn_workspace_fixed_bytes())

    def error_word(self) -> torch.Tensor:
        return self.tensor[:4].view(torch.int32)

    def read_error(self, clear: bool = True, stream=None) -> int:
        error = read_device_error(self.error_word(), clear, stream)
        for tensor in self._before:
            error |= read_device_error(tensor[:4], clear, stream)
        return error


def attn_decode(q, k_cache, v_cache, block_tables, context_lens, scale, out=None, workspace=None,
                num_ctas: int = 0, stream=None):
    """Decode attention through block tables; returns out [B, Hq, 128] bf16."""
    _need(q, torch.bfloat16, "q")
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(v_cache, torch.bfloat16, "v_cache")
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    B, hq, d = q.shape
    nb, hkv, bt, d2 = k_cache.shape
    if d != d2 or v_cache.shape != k_cache.shape or bt not in BLOCK_SIZES:
        raise ValueError("q [B, Hq, D] and caches [NB, Hkv, block_tokens, D] must agree")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.shape != (B,):
        raise ValueError("block_tables must be [B, W] and context_lens [B]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, torch.bfloat16, "out")
    if workspace is None:
        workspace = AttentionWorkspace(B, hkv, device=q.device, stream=stream)
    if bt == BLOCK_TOKENS:
        st = _lib.pkv_attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                  block_tables.shape[1], _ptr(context_lens), B, hq, hkv, d, nb,
                                  float(scale), int(num_ctas), workspace.ptr, workspace.nbytes,
                                  _ptr(out), _stream(stream))
    else:
        st = _lib.pkv_attn_decode_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                     block_tables.shape[1], _ptr(context_lens), B, hq, hkv, d, nb, bt,
                                     float(scale), int(num_ctas), workspace.ptr, workspace.nbytes,
                                     _ptr(out), _stream(stream))
    _check(st, "pkv_attn_decode")
    return out


def attn_decode_cuda_cores(q, k_cache, v_cache, block_tables, context_lens, scale, out=None, workspace=None,
                           num_ctas: int = 0, stream=None):
    """attn_decode with the per-tile math on the FP32 CUDA cores instead of
    the tensor cores (group sizes 4 and 8, 16-token blocks): the measured
    alternative to the tensor-core kernel."""
    _need(q, torch.bfloat16, "q")
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(v_cache, torch.bfloat16, "v_cache")
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    B, hq, d = q.shape
    nb, hkv, bt, d2 = k_cache.shape
    if d != d2 or v_cache.shape != k_cache.shape or bt != BLOCK_TOKENS:
        raise ValueError("q [B, Hq, D] and caches [NB, Hkv, 16, D] must agree")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.shape != (B,):
        raise ValueError("block_tables must be [B, W] and context_lens [B]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, torch.bfloat16, "out")
    if workspace is None:
        workspace = AttentionWorkspace(B, hkv, device=q.device, stream=stream)
    _check(_lib.pkv_attn_decode_cuda_cores(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                           block_tables.shape[1], _ptr(context_lens), B, hq, hkv, d, nb,
                                           float(scale), int(num_ctas), workspace.ptr, workspace.nbytes,
                                           _ptr(out), _stream(stream)),
           "pkv_attn_decode_cuda_cores")
    return out


def decode_step(q, k_new, v_new, slot_mapping, pairs, k_cache, v_cache, block_tables, context_lens, scale,
                out, workspace, device_error=None, num_ctas: int = 0, stream=None):
    """One decode step in one library call: block copies (pairs [n, 2]),
    append of k_new / v_new [B, Hkv, D] at slot_mapping, attention -> out."""
    for t, dt, name in ((q, torch.bfloat16, "q"), (k_new, torch.bfloat16, "k_new"),
                        (v_new, torch.bfloat16, "v_new"), (slot_mapping, torch.int64, "slot_mapping"),
                        (pairs, torch.int32, "pairs"), (k_cache, torch.bfloat16, "k_cache"),
                        (v_cache, torch.bfloat16, "v_cache"), (block_tables, torch.int32, "block_tables"),
                        (context_lens, torch.int32, "context_lens"), (out, torch.bfloat16, "out")):
        _need(t, dt, name)
    B, hq, d = q.shape
    nb, hkv, bt, d2 = k_cache.shape
    T = slot_mapping.numel()
    n = pairs.shape[0] if pairs.numel() else 0
    if d != d2 or v_cache.shape != k_cache.shape or bt != BLOCK_TOKENS or out.shape != q.shape:
        raise ValueError("q/out [B, Hq, D] and caches [NB, Hkv, 16, D] must agree")
    if k_new.shape != (T, hkv, d) or v_new.shape != (T, hkv, d) or (n and pairs.shape != (n, 2)):
        raise ValueError("k_new, v_new must be [T, Hkv, D]; pairs [n, 2]")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.shape != (B,):
        raise ValueError("block_tables must be [B, W] and context_lens [B]")
    _check(_lib.pkv_decode_step(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), T, _ptr(pairs) if n else None, n,
                                _ptr(k_cache), _ptr(v_cache), nb, _ptr(q), _ptr(block_tables),
                                block_tables.shape[1], _ptr(context_lens), B, hq, hkv, d, float(scale),
                                int(num_ctas), workspace.ptr, workspace.nbytes, _ptr(out), _ptr(device_error),
                                _stream(stream)), "pkv_decode_step")
    return out


def step_layout(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_blocks_per_seq: int,
                num_pairs: int = 0) -> dict:
    """Byte offsets (and total size) of a decode step's inputs in one packed buffer."""
    lay = StepLayoutT()
    _check(_lib.pkv_step_layout(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, num_pairs,
                                ctypes.byref(lay)), "pkv_step_layout")
    return {name: int(getattr(lay, name)) for name, _ in StepLayoutT._fields_}


def decode_step_host(host_packed, device_staging, num_pairs, k_cache, v_cache, max_blocks_per_seq, num_seqs,
                     num_q_heads, scale, workspace, device_out, host_out, device_error=None, num_ctas: int = 0,
                     stream=None) -> None:
    """pkv_decode_step_host: the packed inputs (uint8 host tensor) staged into
    device memory -- read across the host link by a kernel when pinned, else
    one copy -- then the step, with the output rows written into host_out
    (directly when pinned, else through device_out and one copy)."""
    _need(host_packed, torch.uint8, "host_packed", cuda=False)
    _need(device_staging, torch.uint8, "device_staging")
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(v_cache, torch.bfloat16, "v_cache")
    _need(device_out, torch.bfloat16, "device_out")
    _need(host_out, torch.bfloat16, "host_out", cuda=False)
    if host_packed.is_cuda or host_out.is_cuda:
        raise ValueError("host_packed and host_out must be host tensors (pinned for asynchronous copies)")
    nb, hkv, bt, d = k_cache.shape
    if bt != BLOCK_TOKENS or v_cache.shape != k_cache.shape:
        raise ValueError("caches must be [NB, Hkv, 16, D] and alike")
    if device_out.shape != (num_seqs, num_q_heads, d) or host_out.shape != device_out.shape:
        raise ValueError("device_out and host_out must be [num_seqs, Hq, D]")
    need = step_layout(num_seqs, num_q_heads, hkv, d, max_blocks_per_seq, num_pairs)["bytes"]
    if host_packed.numel() < need or device_staging.numel() < need:
        raise ValueError(f"packed buffers need {need} bytes")
    _check(_lib.pkv_decode_step_host(_ptr(host_packed), _ptr(device_staging), num_pairs, _ptr(k_cache),
                                     _ptr(v_cache), nb, max_blocks_per_seq, num_seqs, num_q_heads, hkv, d,
                                     float(scale), int(num_ctas), workspace.ptr, workspace.nbytes,
                                     _ptr(device_out), _ptr(host_out), _ptr(device_error), _stream(stream)),
           "pkv_decode_step_host")


class Cascade:
    """Shared-prefix groups of a batch for pkv_attn_decode_cascade: each
    group is (sequence indices of the batch, shared leading blocks). Owns the
    device workspace and the pinned staging of the plan."""

    def __init__(self, num_seqs: int, num_q_heads: int, num_kv_heads: int, groups, device=None, stream=None):
        groups = [(list(map(int, m)), int(sh)) for m, sh in groups]
        self.num_seqs, self.num_q_heads, self.num_kv_heads = num_seqs, num_q_heads, num_kv_heads
        self.groups = groups
        offs = [0]
        for m, _ in groups:
            offs.append(offs[-1] + len(m))
        n = len(groups)
        self._offsets = (ctypes.c_int32 * (n + 1))(*offs)
        self._members = (ctypes.c_int32 * max(1, offs[-1]))(*[x for m, _ in groups for x in m])
        self._shared = (ctypes.c_int32 * max(1, n))(*[sh for _, sh in groups])
        args = (num_seqs, num_q_heads, num_kv_heads, n, self._offsets, self._shared)
        self.nbytes = int(_lib.pkv_attn_cascade_workspace_size(*args))
        staging = int(_lib.pkv_cascade_staging_size(*args))
        if self.nbytes == 0 or staging == 0:
            raise PkvError(PKV_EINVAL, "pkv_attn_cascade_workspace_size")
        self.buffer = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device or "cuda")
        off = (-self.buffer.data_ptr()) % 256
        self.tensor = self.buffer[off: off + self.nbytes]
        self.staging = torch.empty(staging, dtype=torch.uint8).pin_memory()
        _check(_lib.pkv_attn_workspace_init(self.tensor.data_ptr(), self.nbytes, _stream(stream)),
               "pkv_attn_workspace_init")
        _check(_lib.pkv_cascade_plan(num_seqs, num_q_heads, num_kv_heads, n, self._offsets, self._members, self._shared,
                                     self.tensor.data_ptr(), self.nbytes, self.staging.data_ptr(), staging,
                                     _stream(stream)), "pkv_cascade_plan")

    def decode(self, q, k_cache, v_cache, block_tables, context_lens, scale, out=None, stream=None):
        """Decode attention for the batch the groups describe; returns out."""
        _need(q, torch.bfloat16, "q")
        _need(k_cache, torch.bfloat16, "k_cache")
        _need(v_cache, torch.bfloat16, "v_cache")
        _need(block_tables, torch.int32, "block_tables")
        _need(context_lens, torch.int32, "context_lens")
        B, hq, d = q.shape
        nb, hkv, bt, _ = k_cache.shape
        if (B, hq, hkv) != (self.num_seqs, self.num_q_heads, self.num_kv_heads) or bt != BLOCK_TOKENS:
            raise ValueError("batch shape differs from the plan's, or blocks are not 16 tokens")
        if out is None:
            out = torch.empty_like(q)
        _need(out, torch.bfloat16, "out")
        _check(_lib.pkv_attn_decode_cascade(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                            block_tables.shape[1], _ptr(context_lens), B, hq, hkv, d, nb,
                                            float(scale), len(self.groups), self._offsets, self._shared,
                                            self.tensor.data_ptr(), self.nbytes, _ptr(out), _stream(stream)),
               "pkv_attn_decode_cascade")
        return out

    def read_error(self, clear: bool = True, stream=None) -> int:
        """The device error word the three kernels share (then cleared)."""
        return read_device_error(self.tensor[:4].view(torch.int32), clear, stream)


def attn_decode_static(q, k_cache, v_cache, block_tables, context_lens, scale, out, device_error=None,
                       stream=None):
    """attn_decode without a workspace, for callers that cannot allocate:
    the library's own static device scratch is used and nothing is allocated
    (out must be given). Calls on one device must not overlap on the GPU."""
    _need(q, torch.bfloat16, "q")
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(v_cache, torch.bfloat16, "v_cache")
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    _need(out, torch.bfloat16, "out")
    B, hq, d = q.shape
    nb, hkv, bt, d2 = k_cache.shape
    if d != d2 or v_cache.shape != k_cache.shape or bt != BLOCK_TOKENS or out.shape != q.shape:
        raise ValueError("q/out [B, Hq, D] and caches [NB, Hkv, 16, D] must agree")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.shape != (B,):
        raise ValueError("block_tables must be [B, W] and context_lens [B]")
    _check(_lib.pkv_attn_decode_static(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                       block_tables.shape[1], _ptr(context_lens), B, hq, hkv, d, nb,
                                       float(scale), _ptr(device_error), _ptr(out), _stream(stream)),
           "pkv_attn_decode_static")
    return out


# ---------------------------------------------------------------------------
# many query rows per sequence: prompts, draft trees, and the way into the cache


def _need_all(device: int, tensors) -> None:
    """Each (tensor, dtype, name): that dtype, contiguous, on that CUDA device."""
    for t, dtype, name in tensors:
        if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous() or device < 0:
            _need(t, dtype, name)
            raise ValueError(f"{name} is on {t.device}, other tensors on cuda:{device}")


class _LaunchOn:
    """Makes a device current, and `stream` where one is given, so that new
    tensors belong to it; yields the stream's handle."""

    def __init__(self, device: int, stream):
        self.device, self.stream = device, stream

    def __enter__(self) -> int:
        s = self.stream
        if s is not None and not isinstance(s, torch.cuda.Stream):
            s = torch.cuda.ExternalStream(int(s), device=self.device)
        if s is not None and s.device.index != self.device:
            raise ValueError(f"the stream is on {s.device}, the tensors on cuda:{self.device}")
        self.guards = contextlib.ExitStack()
        self.guards.enter_context(torch.cuda.device(self.device))
        if s is None:
            return torch._C._cuda_getCurrentRawStream(self.device)
        self.guards.enter_context(torch.cuda.stream(s))
        return s.cuda_stream

    def __exit__(self, *exc):
        self.guards.close()


class _LaunchHere:
    """The same for the current device and its current stream: nothing to do."""

    def __init__(self, device: int):
        self.device = device

    def __enter__(self) -> int:
        return torch._C._cuda_getCurrentRawStream(self.device)

    def __exit__(self, *exc):
        pass


def _here(device: int, stream) -> int | None:
    """The current stream's handle where that is the one to launch on and `device`
    the current device; None where _LaunchOn has to make them so first."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None and torch._C._cuda_getDevice() == device else None


def _launch_on(device: int, stream):
    if stream is None and torch.cuda.current_device() == device:
        return _LaunchHere(device)
    return _LaunchOn(device, stream)


class PrefillWorkspace:
    """Device scratch for attn_prefill and attn_tree, of any batch (120 MB on 152
    SMs): the error word, then the partial results of rows whose keys are split.
    Its header is zeroed on `stream` (default: the current one); calls on another
    stream wait for that one first, as for any input made there. Calls that share
    a workspace must not overlap on the GPU."""

    def __init__(self, device=None, stream=None):
        dev = torch.device(device or "cuda")
        with torch.cuda.device(dev):
            self.nbytes = int(_lib.pkv_attn_prefill_workspace_size())
            if self.nbytes == 0:
                raise PkvError(PKV_ECUDA, "pkv_attn_prefill_workspace_size")
            self.buffer = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=dev)
            off = (-self.buffer.data_ptr()) % 256
            self.tensor = self.buffer[off : off + self.nbytes]
            self.ptr, self.device = self.tensor.data_ptr(), self.tensor.get_device()
            # only the header has to hold zeros
            _check(_lib.pkv_attn_workspace_init(self.ptr, 256, _stream(stream)), "pkv_attn_workspace_init")

    def read_error(self, clear: bool = True, stream=None) -> int:
        return read_device_error(self.tensor[:4].view(torch.int32), clear, stream)


_BF16, _I32, _I64, _F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


def _rows_shapes(q, k_cache, v_cache, block_tables, context_lens, query_starts, out, workspace):
    device = q.get_device()
    _need_all(device, ((q, _BF16, "q"), (k_cache, _BF16, "k_cache"), (v_cache, _BF16, "v_cache"),
                       (block_tables, _I32, "block_tables"), (context_lens, _I32, "context_lens"),
                       (query_starts, _I32, "query_starts")))
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [T, Hq, D] and caches [NB, Hkv, block_tokens, D]")
    T, hq, d = q.shape
    nb, hkv, bt, d2 = k_cache.shape
    if d != d2 or v_cache.shape != k_cache.shape or bt not in BLOCK_SIZES:
        raise ValueError("q [T, Hq, D] and caches [NB, Hkv, block_tokens in (8, 16, 32, 64), D] must agree")
    if block_tables.dim() != 2 or context_lens.shape != block_tables.shape[:1]:
        raise ValueError("block_tables must be [B, W] and context_lens [B]")
    B, width = block_tables.shape
    if query_starts.dim() != 1 or query_starts.shape[0] != B + 1:
        raise ValueError("query_starts must be [B + 1]")
    if out is not None:
        _need_all(device, ((out, _BF16, "out"),))
        if out.shape != q.shape:
            raise ValueError("out must be shaped like q")
    if workspace is not None and workspace.device != device:
        raise ValueError(f"the workspace is on cuda:{workspace.device}, the tensors on cuda:{device}")
    return device, (T, hq, hkv, d, nb, bt), B, width


def attn_prefill(q, k_cache, v_cache, block_tables, context_lens, query_starts, scale, out=None, workspace=None,
                 stream=None):
    """Causal attention of packed prompt chunks over the cache that holds their
    tokens: rows query_starts[s] .. query_starts[s + 1] of q [T, Hq, 128] are
    the last tokens of sequence s, whose context_lens[s] tokens are all in the
    cache. Returns out [T, Hq, 128]; rows of no sequence are left as they were
    (zeros in an `out` made here). Without a workspace the call makes one for
    itself, and what the device finds wrong (bad block ids, lengths, row starts, a
    wait that ran out) is not reported: pass one and read its read_error()."""
    device, shape, B, width = _rows_shapes(q, k_cache, v_cache, block_tables, context_lens, query_starts, out, workspace)
    with _launch_on(device, stream) as st:
        if out is None:
            out = torch.zeros_like(q)
        if workspace is None:
            workspace = PrefillWorkspace(q.device)
        _check(_lib.pkv_attn_prefill(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
                                     width, context_lens.data_ptr(), query_starts.data_ptr(), B, *shape, float(scale),
                                     workspace.ptr, workspace.nbytes, out.data_ptr(), st), "pkv_attn_prefill")
    return out


def attn_tree(q, k_draft, v_draft, tree_masks, k_cache, v_cache, block_tables, context_lens, query_starts, scale,
              out=None, workspace=None, stream=None):
    """Attention of drafted token trees: draft i (row i of q [T, Hq, 128],
    k_draft, v_draft [T, Hkv, 128], packed by query_starts) sees the
    context_lens[s] tokens of its sequence in the cache and the drafts j of the
    sequence whose bit j is set in tree_masks[i] (int64, see tree_masks()).
    Returns out [T, Hq, 128]; the cache is not written. Without a workspace as
    attn_prefill: device errors are not reported."""
    device, shape, B, width = _rows_shapes(q, k_cache, v_cache, block_tables, context_lens, query_starts, out, workspace)
    _need_all(device, ((k_draft, _BF16, "k_draft"), (v_draft, _BF16, "v_draft"), (tree_masks, _I64, "tree_masks")))
    T, _, hkv, d = shape[:4]
    if k_draft.shape != (T, hkv, d) or v_draft.shape != (T, hkv, d) or tree_masks.shape != (T,):
        raise ValueError("k_draft, v_draft must be [T, Hkv, D] and tree_masks [T]")
    with _launch_on(device, stream) as st:
        if out is None:
            out = torch.zeros_like(q)
        if workspace is None:
            workspace = PrefillWorkspace(q.device)
        _check(_lib.pkv_attn_tree(q.data_ptr(), k_draft.data_ptr(), v_draft.data_ptr(), tree_masks.data_ptr(),
                                  k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), width,
                                  context_lens.data_ptr(), query_starts.data_ptr(), B, *shape, float(scale),
                                  workspace.ptr, workspace.nbytes, out.data_ptr(), st), "pkv_attn_tree")
    return out


def tree_masks(parents) -> list[int]:
    """One sequence's rows of attn_tree's tree_masks from its drafts' parents:
    parents[i] is the index of an earlier draft, or -1 for a draft that follows
    the context. Row i has the bits of i and of its ancestors, as int64 values
    (bit 63 is the sign)."""
    if len(parents) > TREE_MAX_DRAFTS:
        raise ValueError(f"a tree has at most {TREE_MAX_DRAFTS} drafts")
    rows: list[int] = []
    for i, p in enumerate(parents):
        if not -1 <= p < i:
            raise ValueError("a draft's parent is an earlier draft, or -1")
        rows.append((rows[p] if p >= 0 else 0) | (1 << i))
    return [r - (1 << 64) if r >> 63 else r for r in rows]


def rope_table(max_positions: int, rotary_dim: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """cos and sin of every position's angles p * base^(-2 i / rotary_dim), fp32
    [max_positions, rotary_dim] (cosines, then sines), computed in 64 bits: at
    position 100,000 a 32-bit angle is off by up to 0.004."""
    if max_positions < 1 or rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rope_table needs at least one position and an even rotary_dim")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    angle = torch.arange(max_positions, dtype=torch.float64)[:, None] * float(base) ** (-2.0 * i / rotary_dim)
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous().to(device or "cuda")


def _need_rows(device: int, t: torch.Tensor, name: str, T: int, h: int, d: int) -> int:
    """bf16 [T, H, D] whose rows are contiguous; returns the stride of a token."""
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
    if t.shape != (T, h, d):
        raise ValueError(f"{name} must be {[T, h, d]}, got {list(t.shape)}")
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (h > 1 and s1 != d):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    if t.get_device() != device or device < 0:
        raise ValueError(f"{name} is on {t.device}: all tensors must be on one CUDA device")
    return s0 if T > 1 else h * d


def qk_norm_rope_append(q, k, v, cos_sin, positions, slot_mapping, k_cache, v_cache, q_weight=None, k_weight=None,
                        eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None, device_error=None,
                        stream=None):
    """RMS norm of every head of q [T, Hq, D] and k [T, Hkv, D] (skipped where
    the weight is None), rotation by cos_sin[positions] (fp32 [positions,
    rotary_dim], see rope_table(); None: no rotation), and the append of k and
    v to slot_mapping's slots of the caches. q, k, v may be views of one fused
    projection. k_out [T, Hkv, D], where given, receives the normed, rotated
    keys of every row (drafted tokens: slot -1 and k_out). Returns the normed,
    rotated queries [T, Hq, D]."""
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [T, Hq, D] and caches [NB, Hkv, block_tokens, D]")
    device = q.get_device()
    T, hq, d = q.shape
    nb, hkv, bt, d2 = k_cache.shape
    if d != d2 or v_cache.shape != k_cache.shape or bt not in BLOCK_SIZES:
        raise ValueError("q [T, Hq, D] and caches [NB, Hkv, block_tokens in (8, 16, 32, 64), D] must agree")
    qs = _need_rows(device, q, "q", T, hq, d)
    ks = _need_rows(device, k, "k", T, hkv, d)
    vs = _need_rows(device, v, "v", T, hkv, d)
    _need_all(device, ((k_cache, _BF16, "k_cache"), (v_cache, _BF16, "v_cache"), (slot_mapping, _I64, "slot_mapping")))
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [T]")
    qw = kw = cs = ps = None
    if q_weight is not None:
        _need_all(device, ((q_weight, _BF16, "q_weight"),))
        qw = q_weight.data_ptr()
    if k_weight is not None:
        _need_all(device, ((k_weight, _BF16, "k_weight"),))
        kw = k_weight.data_ptr()
    if (qw and q_weight.shape != (d,)) or (kw and k_weight.shape != (d,)):
        raise ValueError("q_weight and k_weight must be [D]")
    max_positions = rotary = 0
    if cos_sin is not None:
        if positions is None:
            raise ValueError("positions must be given with cos_sin")
        _need_all(device, ((cos_sin, _F32, "cos_sin"), (positions, _I32, "positions")))
        if cos_sin.dim() != 2 or positions.shape != (T,):
            raise ValueError("cos_sin must be [positions, rotary_dim] and positions [T]")
        max_positions, rotary = cos_sin.shape
        cs, ps = cos_sin.data_ptr(), positions.data_ptr()
    if q_out is not None:
        _need_all(device, ((q_out, _BF16, "q_out"),))
        if q_out.shape != q.shape:
            raise ValueError("q_out must be shaped like q")
    if k_out is not None:
        _need_all(device, ((k_out, _BF16, "k_out"),))
        if k_out.shape != k.shape:
            raise ValueError("k_out must be shaped like k")
    if device_error is not None:
        _need_all(device, ((device_error, _I32, "device_error"),))
    with _launch_on(device, stream) as st:
        if q_out is None:
            q_out = torch.empty((T, hq, d), dtype=_BF16, device=q.device)
        _check(_lib.pkv_qk_norm_rope_append(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, qw, kw, float(eps), cs,
                                            max_positions, rotary, 1 if interleaved else 0, ps,
                                            slot_mapping.data_ptr(), T, hq, hkv, d, q_out.data_ptr(), _ptr(k_out),
                                            k_cache.data_ptr(), v_cache.data_ptr(), nb, bt, _ptr(device_error), st),
               "pkv_qk_norm_rope_append")
    return q_out


# ---------------------------------------------------------------------------
# a cache held in 4 bits


class Int4Cache:
    """A pool of pages whose keys and values are held in 4 bits (see
    pkv_append_int4 in the header for the format): uint8 `data` [num_blocks, slabs of
    a block, num_kv_heads, bytes of a slab and head], zeros at first. Rows of 128
    values are quantised in groups of group_dims."""

    def __init__(self, num_blocks: int, num_kv_heads: int, block_tokens: int = BLOCK_TOKENS, group_dims: int = 64,
                 device=None):
        nbytes = int(_lib.pkv_int4_block_bytes(num_kv_heads, block_tokens, group_dims))
        if num_blocks < 1 or nbytes == 0:
            raise ValueError("Int4Cache needs blocks, heads, block_tokens in (8, 16, 32, 64) and group_dims in (32, 64, 128)")
        self.num_blocks, self.num_kv_heads = num_blocks, num_kv_heads
        self.block_tokens, self.group_dims = block_tokens, group_dims
        slabs = max(1, block_tokens // 16)
        self._data = torch.zeros((num_blocks, slabs, num_kv_heads, nbytes // slabs // num_kv_heads), dtype=torch.uint8,
                                 device=device or "cuda")
        # of the calls' arguments: the pool's address, and the shape behind it
        self._ptr, self._device = self._data.data_ptr(), self._data.get_device()
        self._shape = num_kv_heads, HEAD_DIM, block_tokens, group_dims

    @property
    def data(self) -> torch.Tensor:
        return self._data


def _need_cache(cache: Int4Cache) -> int:
    if cache._device < 0:
        raise ValueError("the cache must be on a CUDA device")
    return cache._device


def _pairs(pairs) -> int:
    n = pairs.numel()
    if n and (pairs.dim() != 2 or pairs.shape[1] != 2):
        raise ValueError("pairs must be [n, 2]")
    return n // 2


def append_int4(k, v, slot_mapping, cache: Int4Cache, device_error=None, stream=None) -> None:
    """Quantise k[i], v[i] ([T, Hkv, 128] bf16, possibly views of one fused
    projection) into slot slot_mapping[i] (int64; negative: a padding row)."""
    device = _need_cache(cache)
    st = _here(device, stream)
    if st is None:
        with _LaunchOn(device, stream):
            return append_int4(k, v, slot_mapping, cache, device_error)
    tensors, err = ((slot_mapping, _I64, "slot_mapping"),), None
    if device_error is not None:
        tensors, err = tensors + ((device_error, _I32, "device_error"),), device_error.data_ptr()
    _need_all(device, tensors)
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError("k, v must be [T, Hkv, 128]")
    T, (hkv, d, bt, gd) = slot_mapping.numel(), cache._shape
    ks, vs = _need_rows(device, k, "k", T, hkv, d), _need_rows(device, v, "v", T, hkv, d)
    _check(_lib.pkv_append_int4(k.data_ptr(), ks, v.data_ptr(), vs, slot_mapping.data_ptr(), T, cache._ptr, cache.num_blocks,
                                hkv, d, bt, gd, err, st), "pkv_append_int4")


def load_int4(cache: Int4Cache, pairs, k_cache, v_cache, device_error=None, stream=None) -> None:
    """Block pairs[i, 0] of the 4-bit cache as bf16 rows into block pairs[i, 1] of
    k_cache and v_cache [blocks, Hkv, block_tokens, 128]."""
    device = _need_cache(cache)
    st = _here(device, stream)
    if st is None:
        with _LaunchOn(device, stream):
            return load_int4(cache, pairs, k_cache, v_cache, device_error)
    tensors, err = ((k_cache, _BF16, "k_cache"), (v_cache, _BF16, "v_cache"), (pairs, _I32, "pairs")), None
    if device_error is not None:
        tensors, err = tensors + ((device_error, _I32, "device_error"),), device_error.data_ptr()
    _need_all(device, tensors)
    n, (hkv, d, bt, gd), shape = _pairs(pairs), cache._shape, k_cache.shape
    if len(shape) != 4 or shape[1:] != (hkv, bt, d) or v_cache.shape != shape:
        raise ValueError(f"k_cache, v_cache must be {['blocks', hkv, bt, d]} and alike")
    if n:
        _check(_lib.pkv_load_int4(cache._ptr, pairs.data_ptr(), n, k_cache.data_ptr(), v_cache.data_ptr(), cache.num_blocks,
                                  shape[0], hkv, d, bt, gd, err, st), "pkv_load_int4")


def block_copy_int4(cache: Int4Cache, pairs, device_error=None, stream=None) -> None:
    """Copy physical block pairs[i, 0] of the cache onto pairs[i, 1]."""
    device = _need_cache(cache)
    _need_all(device, ((pairs, _I32, "pairs"),))
    if device_error is not None:
        _need_all(device, ((device_error, _I32, "device_error"),))
    n = _pairs(pairs)
    with _launch_on(device, stream) as st:
        _check(_lib.pkv_block_copy_int4(cache._ptr, pairs.data_ptr(), n, cache.num_blocks, *cache._shape, _ptr(device_error),
                                        st), "pkv_block_copy_int4")


def attn_decode_int4(q, cache: Int4Cache, block_tables, context_lens, scale, out=None, workspace=None, num_ctas: int = 0,
                     stream=None):
    """attn_decode over a cache held in 4 bits; returns out [B, Hq, 128] bf16.
    workspace: an AttentionWorkspace (made with int4 where the first call is a
    captured one); without one the call makes it, and device errors are not reported."""
    device = q.get_device()
    _need_all(device, ((q, _BF16, "q"), (block_tables, _I32, "block_tables"), (context_lens, _I32, "context_lens")))
    st = _here(device, stream)
    if st is None:
        with _LaunchOn(device, stream):
            return attn_decode_int4(q, cache, block_tables, context_lens, scale, out, workspace, num_ctas)
    if cache._device != device:
        raise ValueError(f"the cache is on {cache.data.device}, other tensors on cuda:{device}")
    shape, tables = q.shape, block_tables.shape
    if len(shape) != 3 or shape[2] != HEAD_DIM:
        raise ValueError("q must be [B, Hq, 128]")
    B, hq, d = shape
    if len(tables) != 2 or tables[0] != B or context_lens.shape != (B,):
        raise ValueError("block_tables must be [B, W] and context_lens [B]")
    hkv, _, bt, gd = cache._shape
    if out is None:
        out = torch.empty_like(q)
    else:
        _need_all(device, ((out, _BF16, "out"),))
        if out.shape != shape:
            raise ValueError("out must be shaped like q")
    if workspace is None:
        workspace = AttentionWorkspace(B, hkv, device=q.device, int4=True)
    elif workspace.tensor.get_device() != device:
        raise ValueError(f"the workspace is on {workspace.tensor.device}, the tensors on cuda:{device}")
    nbytes = workspace.for_int4(st)
    _check(_lib.pkv_attn_decode_int4(q.data_ptr(), cache._ptr, block_tables.data_ptr(), tables[1], context_lens.data_ptr(), B,
                                     hq, hkv, d, cache.num_blocks, bt, gd, scale, num_ctas, workspace.ptr,
                                     nbytes, out.data_ptr(), st), "pkv_attn_decode_int4")
    return out


# ---------------------------------------------------------------------------
# beam search


class BeamBuffers:
    """What beam_select leaves of each group's `candidates` best continuations,
    best first: scores (fp32), tokens, parents (int32), finished (bool) [groups,
    candidates]; with max_length also lengths (int32) and history (int32 [groups,
    candidates, max_length])."""

    def __init__(self, groups: int, candidates: int, max_length: int = 0, device=None):
        new = lambda dtype, *more: torch.zeros((groups, candidates, *more), dtype=dtype, device=device or "cuda")
        self.shape = groups, candidates, max_length
        self._tensors = [new(_F32), new(_I32), new(_I32), new(torch.bool)]
        self._tensors += [new(_I32), new(_I32, max_length)] if max_length else [None, None]
        self._ptrs, self._device = [_ptr(t) for t in self._tensors], self._tensors[0].get_device()

    scores = property(lambda self: self._tensors[0])
    tokens = property(lambda self: self._tensors[1])
    parents = property(lambda self: self._tensors[2])
    finished = property(lambda self: self._tensors[3])
    lengths = property(lambda self: self._tensors[4])
    history = property(lambda self: self._tensors[5])


class BeamWorkspace:
    """Device scratch of beam_select for one shape; it holds nothing between calls."""

    def __init__(self, groups: int, beams: int, candidates: int, vocab: int, device=None):
        self.shape = groups, beams, candidates, vocab
        self.nbytes = int(_lib.pkv_beam_workspace_size(*self.shape))
        if self.nbytes == 0:
            raise PkvError(PKV_EINVAL, "pkv_beam_workspace_size")
        self.buffer = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device or "cuda")
        off = (-self.buffer.data_ptr()) % 256
        self.tensor = self.buffer[off : off + self.nbytes]
        self.ptr, self.device = self.tensor.data_ptr(), self.tensor.get_device()


def beam_select(logits, scores, finished=None, eos: int = -1, history=None, lengths=None, candidates: int | None = None,
                out: BeamBuffers | None = None, workspace: BeamWorkspace | None = None, device_error=None, stream=None):
    """The best continuations of groups of beams: logits [groups * beams, vocab]
    (bf16 or fp32, rows apart by any stride), scores fp32 [groups, beams]; finished
    bool [groups, beams]; history int32 [groups, beams, max_length] and lengths
    int32 [groups, beams], or neither. Takes out's number of candidates, or
    `candidates` (default: one per beam). Returns the BeamBuffers."""
    device = logits.get_device()
    if logits.dtype not in (_BF16, _F32) or logits.dim() != 2:
        raise ValueError(f"logits must be bf16 or fp32 [groups * beams, vocab], got {logits.dtype} {list(logits.shape)}")
    _need_all(device, ((scores, _F32, "scores"),))
    st = _here(device, stream)
    if st is None:
        with _LaunchOn(device, stream):
            return beam_select(logits, scores, finished, eos, history, lengths, candidates, out, workspace, device_error)
    rows, vocab = logits.shape
    shape = scores.shape
    if len(shape) != 2 or rows != shape[0] * shape[1] or rows == 0:
        raise ValueError("scores must be [groups, beams], a row of logits each")
    groups, beams = shape
    if vocab > 1 and logits.stride(1) != 1:
        raise ValueError("a row of logits must be contiguous")
    if finished is not None:
        _need_all(device, ((finished, torch.bool, "finished"),))
        if finished.shape != shape:
            raise ValueError("finished must be shaped like scores")
    if (history is None) != (lengths is None):
        raise ValueError("history and lengths come together")
    room = 0
    if history is not None:
        _need_all(device, ((history, _I32, "history"), (lengths, _I32, "lengths")))
        if history.dim() != 3 or history.shape[:2] != shape or lengths.shape != shape or history.shape[2] < 1:
            raise ValueError("history must be [groups, beams, max_length] and lengths [groups, beams]")
        room = history.shape[2]
    n = candidates if candidates is not None else out.shape[1] if out is not None else beams
    if out is not None:
        if out._device != device or out.shape[:2] != (groups, n):
            raise ValueError(f"out must hold {groups} groups of {n} candidates on cuda:{device}")
        if room and out.shape[2] != room:
            raise ValueError("out's histories must be [groups, candidates, max_length], as the beams'")
        if out._ptrs[0] == scores.data_ptr():
            raise ValueError("out must not be the beams' own buffers")
    if workspace is not None and workspace.device != device:
        raise ValueError(f"the workspace is on cuda:{workspace.device}, the tensors on cuda:{device}")
    if device_error is not None:
        _need_all(device, ((device_error, _I32, "device_error"),))
    if out is None:
        out = BeamBuffers(groups, n, room, device=logits.device)
    if workspace is None:
        workspace = BeamWorkspace(groups, beams, n, vocab, device=logits.device)
    so, to, po, fo, lo, ho = out._ptrs
    _check(_lib.pkv_beam_select(logits.data_ptr(), logits.stride(0) if rows > 1 else vocab, 2 if logits.dtype is _BF16 else 4,
                                scores.data_ptr(), _ptr(finished), eos, groups, beams, n, vocab, _ptr(history), _ptr(lengths),
                                room, so, to, po, fo, lo if room else None, ho if room else None, workspace.ptr,
                                workspace.nbytes, _ptr(device_error), st), "pkv_beam_select")
    return out


# ---------------------------------------------------------------------------
# host block manager


class BlockManager:
    """Free list, refcounts, copy-on-write, page-rounded admission, incremental
    allocation with preemption, and the prefix-cache index (C++)."""

    def __init__(self, num_blocks: int, block_tokens: int = BLOCK_TOKENS, free_order=None,
                 incremental: bool = False, watermark: int = 0, prefix_cache: bool = False):
        order = None
        self._order_buf = None
        if free_order is not None:
            arr = (ctypes.c_int32 * num_blocks)(*[int(x) for x in free_order])
            self._order_buf = arr
            order = ctypes.cast(arr, ctypes.c_void_p)
        self._h = _lib.pkv_bm_create_ex(num_blocks, block_tokens, order, int(incremental), watermark,
                                        int(prefix_cache))
        if not self._h:
            raise PkvError(PKV_EINVAL, "pkv_bm_create_ex")
        self.num_blocks, self.block_tokens = num_blocks, block_tokens
        self.reused: dict[int, int] = {}
        # a sequence's prompt tokens, and how many of them from the first on are in
        # their slots or on their way (the engine counts these)
        self.prompt: dict[int, int] = {}
        self.written: dict[int, int] = {}

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _lib.pkv_bm_destroy(h)
            self._h = None

    def admit(self, prompt_len: int, max_new: int, group: int = -1, prefix_len: int = 0, tokens=None) -> int:
        """tokens (the prompt's ids) selects pkv_bm_admit_tokens; the number of
        reused cached blocks is then kept in self.reused[seq_id]."""
        sid = ctypes.c_int(0)
        if tokens is None:
            _check(_lib.pkv_bm_admit(self._h, prompt_len, max_new, group, prefix_len, ctypes.byref(sid)),
                   "pkv_bm_admit")
            self.reused[sid.value], self.prompt[sid.value], self.written[sid.value] = 0, prompt_len, 0
            return sid.value
        if group >= 0 or len(tokens) != prompt_len:
            raise PkvError(PKV_EINVAL, "pkv_bm_admit_tokens: no group, one token per prompt position")
        buf = (ctypes.c_int32 * max(prompt_len, 1))(*[int(t) for t in tokens])
        reused = ctypes.c_int(0)
        _check(_lib.pkv_bm_admit_tokens(self._h, buf, prompt_len, max_new, ctypes.byref(sid),
                                        ctypes.byref(reused)), "pkv_bm_admit_tokens")
        self.reused[sid.value], self.prompt[sid.value] = reused.value, prompt_len
        self.written[sid.value] = reused.value * self.block_tokens
        return sid.value

    def fork(self, parent: int, n: int) -> list[int]:
        ids = (ctypes.c_int32 * max(n, 1))()
        _check(_lib.pkv_bm_fork(self._h, parent, n, ids), "pkv_bm_fork")
        for i in ids[:n]:
            self.prompt[i], self.written[i] = self.prompt[parent], self.written[parent]
        return list(ids[:n])

    def reorder(self, seq_ids, parents) -> None:
        """Sequence seq_ids[i] goes on as seq_ids[parents[i]] is now (beam search):
        tables are shared by reference; PoolExhausted leaves all as it was."""
        n = len(seq_ids)
        if len(parents) != n:
            raise ValueError("one parent per sequence")
        ids = (ctypes.c_int32 * max(n, 1))(*[int(x) for x in seq_ids])
        src = (ctypes.c_int32 * max(n, 1))(*[int(x) for x in parents])
        _check(_lib.pkv_bm_reorder(self._h, ids, src, n), "pkv_bm_reorder")
        for kept in (self.prompt, self.written):
            was = [kept[s] for s in ids[:n]]
            kept.update({s: was[p] for s, p in zip(ids[:n], src[:n])})

    def prepare_append(self, seq_ids):
        """Returns (slots list[int], pairs list[(src, dst)])."""
        n = len(seq_ids)
        ids = (ctypes.c_int32 * max(n, 1))(*seq_ids)
        slots = (ctypes.c_int64 * max(n, 1))()
        pairs = (ctypes.c_int32 * max(2 * n, 2))()
        npairs = ctypes.c_int(0)
        _check(_lib.pkv_bm_prepare_append(self._h, ids, n, slots, pairs, ctypes.byref(npairs)),
               "pkv_bm_prepare_append")
        return list(slots[:n]), [(pairs[2 * i], pairs[2 * i + 1]) for i in range(npairs.value)]

    def free(self, seq_id: int) -> None:
        _check(_lib.pkv_bm_free(self._h, seq_id), "pkv_bm_free")
        for kept in (self.reused, self.prompt, self.written):
            kept.pop(seq_id, None)

    def preempt(self, seq_id: int) -> int:
        n = ctypes.c_int(0)
        _check(_lib.pkv_bm_preempt(self._h, seq_id, ctypes.byref(n)), "pkv_bm_preempt")
        # all its tokens are to be recomputed
        self.prompt[seq_id], self.written[seq_id] = self.context_len(seq_id), 0
        return n.value

    def resume(self, seq_id: int) -> None:
        _check(_lib.pkv_bm_resume(self._h, seq_id), "pkv_bm_resume")

    def newest_running(self) -> int:
        return int(_lib.pkv_bm_newest_running(self._h))

    def slots(self, seq_id: int, first: int, n: int) -> list[int]:
        buf = (ctypes.c_int64 * max(n, 1))()
        _check(_lib.pkv_bm_slots(self._h, seq_id, first, n, buf), "pkv_bm_slots")
        return list(buf[:n])

    def table(self, seq_id: int) -> list[int]:
        length = ctypes.c_int(0)
        st = _lib.pkv_bm_block_table(self._h, seq_id, None, 0, ctypes.byref(length))
        if st not in (PKV_OK, PKV_ERANGE):
            _check(st, "pkv_bm_block_table")
        buf = (ctypes.c_int32 * max(length.value, 1))()
        _check(_lib.pkv_bm_block_table(self._h, seq_id, buf, length.value, ctypes.byref(length)),
               "pkv_bm_block_table")
        return list(buf[: length.value])

    def context_len(self, seq_id: int) -> int:
        c = ctypes.c_int(0)
        _check(_lib.pkv_bm_context_len(self._h, seq_id, ctypes.byref(c)), "pkv_bm_context_len")
        return c.value

    def batch_tables(self, seq_ids, width: int):
        """(tables int32 [n, width] with -1 padding, context_lens int32 [n]) as CPU tensors."""
        n = len(seq_ids)
        ids = (ctypes.c_int32 * max(n, 1))(*seq_ids)
        tables = torch.empty((n, width), dtype=torch.int32)
        ctx = torch.empty((n,), dtype=torch.int32)
        _check(_lib.pkv_bm_batch_tables(self._h, ids, n, tables.data_ptr(), width, ctx.data_ptr()),
               "pkv_bm_batch_tables")
        return tables, ctx

    def stats(self) -> dict:
        s = StatsT()
        _check(_lib.pkv_bm_stats(self._h, ctypes.byref(s)), "pkv_bm_stats")
        return {"free": s.free_blocks, "used": s.used_blocks, "shared": s.shared_blocks,
                "ref_sum": s.ref_sum, "spares": s.spare_blocks, "cow_copies": s.cow_copies,
                "seqs": s.num_seqs, "cached": s.cached_blocks, "cached_idle": s.cached_idle_blocks,
                "available": s.available_blocks, "cache_hits": s.cache_hits, "evictions": s.evictions,
                "preempted": s.preempted_seqs}

    def refcount(self, block: int) -> int:
        return int(_lib.pkv_bm_refcount(self._h, block))
