"""GB300-native speculative-decoding verification sampler.

Python binding of the C ABI in ``include/spec_verify.h`` (``libspecverify.so``, built in-tree
for sm_103a by :func:`build`). This module only marshals arguments: every step of the
verification runs in the library's CUDA kernels. PyTorch tensors are accepted for device
memory and streams; raw integer pointers work as well.

The same names as the C ABI are exported (``spec_verify_init``, ``spec_verify_run``, ...),
plus :class:`SpecVerify`, a small owner of a context.
"""
from __future__ import annotations

import ctypes
import os
import re
import subprocess
import tempfile

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
_INCLUDE = os.path.join(_ROOT, "include")
_HEADER = os.path.join(_INCLUDE, "spec_verify.h")
_UNITS = [os.path.join(_PKG, "csrc", f) for f in ("spec_verify.cu", "sv_rows.cu", "sv_cache.cu")]
_SOURCES = [*_UNITS, *(os.path.join(_PKG, "csrc", f) for f in ("sv_device.cuh", "sv_rows.cuh",
                                                                "sv_rows_block.cuh", "sv_cache.cuh",
                                                                "sv_cache_attention.cuh"))]
# SPEC_VERIFY_DEBUG_BOUNDS=1 in the environment selects the checked build (-DSV_DEBUG_BOUNDS): every
# global load and store of the kernels is checked against the call's arrays, and an access
# outside them is skipped and reported as SV_ERR_BOUNDS in the error word (by the row and cache operators in
# those that spec_verify_rows_outside and spec_verify_cache_outside of that build read). For tests only.
DEBUG_BOUNDS = os.environ.get("SPEC_VERIFY_DEBUG_BOUNDS", "0") not in ("", "0")
RELEASE_LIB_PATH = os.path.join(_PKG, "libspecverify.so")
DEBUG_LIB_PATH = os.path.join(_PKG, "libspecverify_debug.so")
LIB_PATH = DEBUG_LIB_PATH if DEBUG_BOUNDS else RELEASE_LIB_PATH

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-shared", "-Xcompiler", "-fPIC", "--threads", "3", "-I" + _INCLUDE]

SV_OK, SV_EINVAL, SV_ECAPACITY, SV_EDTYPE, SV_ECUDA, SV_EDEVICE = 0, -1, -2, -3, -4, -5
SV_F32, SV_BF16, SV_F16, SV_E4M3 = 0, 1, 2, 3
SV_DRAFT_PROBS, SV_DRAFT_LOGITS = 1, 2
SV_MAX_SYNTHETIC = 64
SV_ROWS_MAX_VOCAB, SV_MAX_TOP = 524288, 64
SV_MAX_HEAD_DIM, SV_MAX_AXES, SV_MAX_PAGE, SV_CACHE_WORKSPACE = 256, 4, 65536, 10121984


class Batch(ctypes.Structure):
    """spec_verify_batch of include/spec_verify.h."""
    _fields_ = [("logits", ctypes.c_void_p), ("draft_ids", ctypes.c_void_p),
                ("draft_probs", ctypes.c_void_p), ("draft_logits", ctypes.c_void_p),
                ("cu_num_draft", ctypes.c_void_p), ("temperature", ctypes.c_void_p),
                ("is_greedy", ctypes.c_void_p), ("partial_prefill", ctypes.c_void_p),
                ("frequency_penalty", ctypes.c_void_p), ("output_bin_counts", ctypes.c_void_p),
                ("counts_row", ctypes.c_void_p), ("top_k", ctypes.c_void_p),
                ("top_p", ctypes.c_void_p),
                ("seed", ctypes.c_uint64), ("req_index_base", ctypes.c_uint32),
                ("num_reqs", ctypes.c_int32), ("num_draft_tokens", ctypes.c_int32),
                ("max_spec_len_this_batch", ctypes.c_int32), ("counts_rows", ctypes.c_int32),
                ("fp64_gumbel", ctypes.c_int32)]


class Outputs(ctypes.Structure):
    """spec_verify_outputs of include/spec_verify.h."""
    _fields_ = [("sampled", ctypes.c_void_p), ("num_sampled", ctypes.c_void_p),
                ("num_rejected", ctypes.c_void_p), ("row_max", ctypes.c_void_p),
                ("row_sumexp", ctypes.c_void_p), ("row_argmax", ctypes.c_void_p)]


class SampleArgs(ctypes.Structure):
    """spec_verify_sample_args of include/spec_verify.h."""
    _fields_ = [("logits", ctypes.c_void_p), ("logits_stride", ctypes.c_int64),
                ("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p),
                ("top_p", ctypes.c_void_p), ("min_p", ctypes.c_void_p),
                ("uniforms", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
                ("token_logprob", ctypes.c_void_p), ("probs", ctypes.c_void_p),
                ("probs_stride", ctypes.c_int64), ("num_rows", ctypes.c_int32),
                ("vocab_size", ctypes.c_int32), ("logits_dtype", ctypes.c_int32),
                ("device", ctypes.c_int32)]


class LogprobsArgs(ctypes.Structure):
    """spec_verify_logprobs_args of include/spec_verify.h."""
    _fields_ = [("logits", ctypes.c_void_p), ("logits_stride", ctypes.c_int64),
                ("temperature", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
                ("cu_num_draft", ctypes.c_void_p), ("token_logprob", ctypes.c_void_p),
                ("token_rank", ctypes.c_void_p), ("top_ids", ctypes.c_void_p),
                ("top_logprobs", ctypes.c_void_p), ("token_stride", ctypes.c_int32),
                ("num_reqs", ctypes.c_int32), ("num_top", ctypes.c_int32),
                ("num_rows", ctypes.c_int32), ("vocab_size", ctypes.c_int32),
                ("logits_dtype", ctypes.c_int32), ("device", ctypes.c_int32)]


_VP, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class CacheAppendArgs(ctypes.Structure):
    """spec_verify_cache_append_args of include/spec_verify.h."""
    _fields_ = [*((f, _VP) for f in ("q", "k", "v", "q_out", "k_cache", "v_cache")),
                *((f, _I64) for f in ("q_row_stride", "q_head_stride", "k_row_stride", "k_head_stride",
                                      "v_row_stride", "v_head_stride", "q_out_row_stride", "q_out_head_stride",
                                      "k_page_stride", "k_slot_stride", "k_cache_head_stride",
                                      "v_page_stride", "v_slot_stride", "v_cache_head_stride")),
                ("page_table", _VP), ("table_stride", _I64), ("lengths", _VP), ("cu_num_draft", _VP),
                ("positions", _VP), ("positions_stride", _I64), ("inv_freq", _VP), ("k_scale", _VP),
                ("v_scale", _VP), ("axes", ctypes.c_char_p),
                *((f, _I32) for f in ("num_rows", "num_reqs", "num_q_heads", "num_kv_heads", "head_dim",
                                      "rotary_dim", "interleaved", "num_axes", "num_pages", "page_size",
                                      "pages_per_req", "dtype", "cache_dtype", "device"))]


class CacheAttentionArgs(ctypes.Structure):
    """spec_verify_cache_attention_args of include/spec_verify.h."""
    _fields_ = [*((f, _VP) for f in ("q", "k_cache", "v_cache", "out", "lse")),
                *((f, _I64) for f in ("q_row_stride", "q_head_stride", "out_row_stride", "out_head_stride",
                                      "k_page_stride", "k_slot_stride", "k_cache_head_stride",
                                      "v_page_stride", "v_slot_stride", "v_cache_head_stride")),
                ("page_table", _VP), ("table_stride", _I64), ("lengths", _VP), ("cu_num_draft", _VP),
                ("k_scale", _VP), ("v_scale", _VP), ("workspace", _VP), ("workspace_bytes", _I64),
                ("scale", ctypes.c_float),
                *((f, _I32) for f in ("window", "num_rows", "num_reqs", "num_q_heads", "num_kv_heads",
                                      "head_dim", "num_pages", "page_size", "pages_per_req", "dtype",
                                      "cache_dtype", "device"))]


SV_ERR_BATCH, SV_ERR_COUNTS, SV_ERR_BOUNDS, SV_ERR_SELECT, SV_ERR_WAIT = 1, 2, 4, 8, 16
KERNELS = ("stats", "verify", "select")  # profiling slots (select: top-k / top-p calls)

_lib = None


class SpecVerifyError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = _status_string(status)
        super().__init__(f"{what}: {msg} ({status})")
        self.status = status


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _stale(path: str | None = None) -> bool:
    path = path or LIB_PATH
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(s) > t for s in _SOURCES + [_HEADER])


def build(force: bool = False, verbose: bool = False, debug: bool | None = None) -> str:
    """Compile libspecverify.so (or, with debug=True, the checked libspecverify_debug.so) for
    sm_103a next to this file (atomic replace). debug=None: the build this process loads."""
    debug = DEBUG_BOUNDS if debug is None else debug
    path = DEBUG_LIB_PATH if debug else RELEASE_LIB_PATH
    if not force and not _stale(path):
        return path
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=_PKG)
    os.close(fd)
    cmd = [_nvcc(), *NVCC_FLAGS, *(["-DSV_DEBUG_BOUNDS"] if debug else []), "-o", tmp, *_UNITS]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stderr[-4000:])
        if verbose:
            print(r.stderr)
        os.replace(tmp, path)
    finally:
        if os.path.exists(tmp):
            os.unlink(tmp)
    return path


def build_all(force: bool = False) -> None:
    """Both builds (the library and its checked debug variant), compiled in parallel."""
    import threading

    errors = []

    def one(debug):
        try:
            build(force=force, debug=debug)
        except Exception as e:  # noqa: BLE001 - re-raised below
            errors.append(e)

    threads = [threading.Thread(target=one, args=(d,)) for d in (False, True)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


def declared_symbols() -> list[str]:
    """Names of the functions include/spec_verify.h declares."""
    with open(_HEADER, encoding="utf-8") as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(spec_verify_\w+)\s*\(", text, re.M)))


def lib():
    """The loaded C library (ctypes), built first if missing. Raises if it cannot be built or
    loaded: there is no fallback implementation."""
    global _lib
    if _lib is not None:
        return _lib
    if _stale():
        # a library older than its sources is never loaded: a failed rebuild raises, so that a
        # compile error cannot leave the previous binary running (and measured) in its place
        try:
            build()
        except (OSError, RuntimeError) as e:
            raise RuntimeError("libspecverify.so is out of date and could not be rebuilt: "
                               + str(e)) from e
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, u32, u64, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int64
    L.spec_verify_init.argtypes = [ctypes.POINTER(vp), i32, i32, i32, i32, i32, i32]
    L.spec_verify_run.argtypes = [vp, vp, vp, vp, vp, vp, vp, u64, u32, i32, i32, i32, vp, vp, vp,
                                  vp, vp, vp, vp]
    L.spec_verify_run_draft_logits.argtypes = list(L.spec_verify_run.argtypes)
    L.spec_verify_run_batch.argtypes = [vp, ctypes.POINTER(Batch), ctypes.POINTER(Outputs), vp]
    L.spec_verify_set_synthetic.argtypes = [vp, vp, i32]
    L.spec_verify_shard_stats.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp]
    L.spec_verify_shard_race.argtypes = [vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, u64, u32,
                                         i32, i32, i32, vp, vp]
    L.spec_verify_shard_finish.argtypes = [vp, vp, i32, vp, vp, i32, i32, vp, vp, vp, vp]
    L.spec_verify_synthetic_rates.argtypes = [ctypes.c_double, i32, vp]
    L.spec_verify_run_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, u64, u32, i32, i32, i32, vp, vp,
                                       vp, vp]
    L.spec_verify_run_noalloc.argtypes = [vp, i32, i32, vp, vp, vp, vp, vp, u64, u32, i32, i32,
                                          i32, vp, vp, vp, vp, vp, vp, vp]
    L.spec_verify_noalloc_last_error.argtypes = [ctypes.POINTER(u32)]
    L.spec_verify_sample.argtypes = [ctypes.POINTER(SampleArgs), vp]
    L.spec_verify_logprobs.argtypes = [ctypes.POINTER(LogprobsArgs), vp]
    L.spec_verify_cache_append.argtypes = [ctypes.POINTER(CacheAppendArgs), vp]
    L.spec_verify_cache_attention.argtypes = [ctypes.POINTER(CacheAttentionArgs), vp]
    L.spec_verify_cache_attention_workspace.argtypes = [ctypes.POINTER(CacheAttentionArgs),
                                                        ctypes.POINTER(i64)]
    L.spec_verify_cache_last_error.argtypes = [ctypes.POINTER(u32)]
    L.spec_verify_reserve_host_io.argtypes = [vp]
    L.spec_verify_last_error.argtypes = [vp, ctypes.POINTER(u32)]
    L.spec_verify_set_profiling.argtypes = [vp, i32]
    L.spec_verify_get_profile.argtypes = [vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64)]
    L.spec_verify_set_chunks.argtypes = [vp, i32]
    L.spec_verify_launches_per_run.argtypes = []
    L.spec_verify_free.argtypes = [vp]
    L.spec_verify_free.restype = None
    L.spec_verify_status_string.argtypes = [i32]
    L.spec_verify_status_string.restype = ctypes.c_char_p
    for f in ("spec_verify_init", "spec_verify_run", "spec_verify_run_draft_logits",
              "spec_verify_run_batch", "spec_verify_set_synthetic", "spec_verify_synthetic_rates",
              "spec_verify_shard_stats", "spec_verify_shard_race", "spec_verify_shard_finish",
              "spec_verify_run_host", "spec_verify_run_noalloc", "spec_verify_noalloc_last_error",
              "spec_verify_sample", "spec_verify_logprobs", "spec_verify_cache_append",
              "spec_verify_cache_attention", "spec_verify_cache_attention_workspace",
              "spec_verify_cache_last_error",
              "spec_verify_reserve_host_io", "spec_verify_last_error", "spec_verify_set_profiling",
              "spec_verify_get_profile", "spec_verify_set_chunks", "spec_verify_launches_per_run"):
        getattr(L, f).restype = i32
    _lib = L
    return L


def _status_string(status: int) -> str:
    try:
        return lib().spec_verify_status_string(status).decode()
    except Exception:  # noqa: BLE001 - only for messages
        return "status"


def _check(status: int, what: str) -> None:
    if status != SV_OK:
        raise SpecVerifyError(status, what)


def _ptr(x):
    """Device or host address of a tensor / array / int (None -> NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if not x.is_contiguous():
            raise ValueError("tensors must be contiguous")
        return x.data_ptr()
    if hasattr(x, "ctypes"):
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x)}")


def _stream_handle(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---- thin wrappers with the C names --------------------------------------------------------

def spec_verify_init(max_num_reqs: int, max_spec_len: int, vocab_size: int, logits_dtype: int,
                     draft_input: int, device: int) -> int:
    ctx = ctypes.c_void_p()
    _check(lib().spec_verify_init(ctypes.byref(ctx), max_num_reqs, max_spec_len, vocab_size,
                                  logits_dtype, draft_input, device), "spec_verify_init")
    return ctx.value


def spec_verify_run(ctx, logits, draft_ids, draft_probs, cu_num_draft, temperature, is_greedy,
                    seed, req_index_base, num_reqs, num_draft_tokens, max_spec_len_this_batch,
                    sampled, num_sampled, num_rejected, opt_row_max=None, opt_row_sumexp=None,
                    opt_row_argmax=None, cuda_stream=None) -> None:
    _check(lib().spec_verify_run(ctx, _ptr(logits), _ptr(draft_ids), _ptr(draft_probs),
                                 _ptr(cu_num_draft), _ptr(temperature), _ptr(is_greedy), seed,
                                 req_index_base, num_reqs, num_draft_tokens,
                                 max_spec_len_this_batch, _ptr(sampled), _ptr(num_sampled),
                                 _ptr(num_rejected), _ptr(opt_row_max), _ptr(opt_row_sumexp),
                                 _ptr(opt_row_argmax), _stream_handle(cuda_stream)),
           "spec_verify_run")


def spec_verify_run_draft_logits(ctx, logits, draft_ids, draft_logits, cu_num_draft, temperature,
                                 is_greedy, seed, req_index_base, num_reqs, num_draft_tokens,
                                 max_spec_len_this_batch, sampled, num_sampled, num_rejected,
                                 opt_row_max=None, opt_row_sumexp=None, opt_row_argmax=None,
                                 cuda_stream=None) -> None:
    _check(lib().spec_verify_run_draft_logits(
        ctx, _ptr(logits), _ptr(draft_ids), _ptr(draft_logits), _ptr(cu_num_draft),
        _ptr(temperature), _ptr(is_greedy), seed, req_index_base, num_reqs, num_draft_tokens,
        max_spec_len_this_batch, _ptr(sampled), _ptr(num_sampled), _ptr(num_rejected),
        _ptr(opt_row_max), _ptr(opt_row_sumexp), _ptr(opt_row_argmax),
        _stream_handle(cuda_stream)), "spec_verify_run_draft_logits")


def spec_verify_run_batch(ctx, batch: Batch, out: Outputs, cuda_stream=None) -> None:
    _check(lib().spec_verify_run_batch(ctx, ctypes.byref(batch), ctypes.byref(out),
                                       _stream_handle(cuda_stream)), "spec_verify_run_batch")


def spec_verify_set_synthetic(ctx, rates) -> None:
    """rates: host sequence of unconditional per-position acceptance rates ([] = off)."""
    import numpy as np
    r = np.ascontiguousarray(np.asarray(rates, dtype=np.float32).reshape(-1))
    _check(lib().spec_verify_set_synthetic(ctx, r.ctypes.data if r.size else None, r.size),
           "spec_verify_set_synthetic")


def spec_verify_synthetic_rates(mean_length: float, num_spec: int):
    """Minimum-variance per-position rates for a target mean accepted length (numpy float32)."""
    import numpy as np
    out = np.zeros(max(num_spec, 0), dtype=np.float32)
    _check(lib().spec_verify_synthetic_rates(float(mean_length), num_spec,
                                             out.ctypes.data if out.size else None),
           "spec_verify_synthetic_rates")
    return out


SHARD_RECORD_BYTES = 24  # spec_verify_shard_stat and spec_verify_shard_key


def spec_verify_shard_stats(ctx, logits_shard, v0, draft_ids, draft_probs_shard, cu_num_draft,
                            temperature, is_greedy, num_reqs, num_draft_tokens,
                            max_spec_len_this_batch, out, cuda_stream=None) -> None:
    _check(lib().spec_verify_shard_stats(ctx, _ptr(logits_shard), v0, _ptr(draft_ids),
                                         _ptr(draft_probs_shard), _ptr(cu_num_draft),
                                         _ptr(temperature), _ptr(is_greedy), num_reqs,
                                         num_draft_tokens, max_spec_len_this_batch, _ptr(out),
                                         _stream_handle(cuda_stream)), "spec_verify_shard_stats")


def spec_verify_shard_race(ctx, logits_shard, v0, vocab_size, all_stats, world, draft_ids,
                           draft_probs_shard, cu_num_draft, temperature, is_greedy, seed,
                           req_index_base, num_reqs, num_draft_tokens, max_spec_len_this_batch,
                           out, cuda_stream=None) -> None:
    _check(lib().spec_verify_shard_race(ctx, _ptr(logits_shard), v0, vocab_size, _ptr(all_stats),
                                        world, _ptr(draft_ids), _ptr(draft_probs_shard),
                                        _ptr(cu_num_draft), _ptr(temperature), _ptr(is_greedy),
                                        seed, req_index_base, num_reqs, num_draft_tokens,
                                        max_spec_len_this_batch, _ptr(out),
                                        _stream_handle(cuda_stream)), "spec_verify_shard_race")


def spec_verify_shard_finish(ctx, all_races, world, draft_ids, cu_num_draft, num_reqs,
                             max_spec_len_this_batch, sampled, num_sampled, num_rejected,
                             cuda_stream=None) -> None:
    _check(lib().spec_verify_shard_finish(ctx, _ptr(all_races), world, _ptr(draft_ids),
                                          _ptr(cu_num_draft), num_reqs, max_spec_len_this_batch,
                                          _ptr(sampled), _ptr(num_sampled), _ptr(num_rejected),
                                          _stream_handle(cuda_stream)), "spec_verify_shard_finish")


def spec_verify_run_host(ctx, logits, draft_ids, draft_probs, cu_num_draft, temperature,
                         is_greedy, seed, req_index_base, num_reqs, num_draft_tokens,
                         max_spec_len_this_batch, sampled, num_sampled, num_rejected,
                         cuda_stream=None) -> None:
    _check(lib().spec_verify_run_host(ctx, _ptr(logits), _ptr(draft_ids), _ptr(draft_probs),
                                      _ptr(cu_num_draft), _ptr(temperature), _ptr(is_greedy), seed,
                                      req_index_base, num_reqs, num_draft_tokens,
                                      max_spec_len_this_batch, _ptr(sampled), _ptr(num_sampled),
                                      _ptr(num_rejected), _stream_handle(cuda_stream)),
           "spec_verify_run_host")


def spec_verify_run_noalloc(logits, logits_dtype, vocab_size, draft_ids, draft_probs,
                            cu_num_draft, temperature, is_greedy, seed, req_index_base, num_reqs,
                            num_draft_tokens, max_spec_len_this_batch, sampled, num_sampled,
                            num_rejected, opt_row_max=None, opt_row_sumexp=None,
                            opt_row_argmax=None, cuda_stream=None) -> None:
    """Verification that allocates nothing (scratch in a static device array of the library,
    limits SV_NOALLOC_MAX_*), for callers that cannot allocate device memory. Runs on the
    current device; overlapping calls on one device race and must be serialised."""
    _check(lib().spec_verify_run_noalloc(_ptr(logits), _dtype_code(logits_dtype)
                                         if isinstance(logits_dtype, str) else logits_dtype,
                                         vocab_size, _ptr(draft_ids), _ptr(draft_probs),
                                         _ptr(cu_num_draft), _ptr(temperature), _ptr(is_greedy),
                                         seed, req_index_base, num_reqs, num_draft_tokens,
                                         max_spec_len_this_batch, _ptr(sampled), _ptr(num_sampled),
                                         _ptr(num_rejected), _ptr(opt_row_max),
                                         _ptr(opt_row_sumexp), _ptr(opt_row_argmax),
                                         _stream_handle(cuda_stream)),
           "spec_verify_run_noalloc")


def spec_verify_noalloc_last_error() -> int:
    """Read and clear the error word of spec_verify_run_noalloc on the current device (waits
    for the device)."""
    w = ctypes.c_uint32()
    _check(lib().spec_verify_noalloc_last_error(ctypes.byref(w)), "spec_verify_noalloc_last_error")
    return w.value


def spec_verify_sample(args: SampleArgs, cuda_stream=None) -> None:
    _check(lib().spec_verify_sample(ctypes.byref(args), _stream_handle(cuda_stream)),
           "spec_verify_sample")


def spec_verify_logprobs(args: LogprobsArgs, cuda_stream=None) -> None:
    _check(lib().spec_verify_logprobs(ctypes.byref(args), _stream_handle(cuda_stream)),
           "spec_verify_logprobs")


def spec_verify_cache_append(args: CacheAppendArgs, cuda_stream=None) -> None:
    _check(lib().spec_verify_cache_append(ctypes.byref(args), _stream_handle(cuda_stream)),
           "spec_verify_cache_append")


def spec_verify_cache_attention(args: CacheAttentionArgs, cuda_stream=None) -> None:
    _check(lib().spec_verify_cache_attention(ctypes.byref(args), _stream_handle(cuda_stream)),
           "spec_verify_cache_attention")


def spec_verify_cache_attention_workspace(args: CacheAttentionArgs) -> int:
    """Bytes of workspace that spec_verify_cache_attention needs for arguments of these sizes and types."""
    n = ctypes.c_int64()
    _check(lib().spec_verify_cache_attention_workspace(ctypes.byref(args), ctypes.byref(n)),
           "spec_verify_cache_attention_workspace")
    return n.value


def spec_verify_cache_last_error() -> int:
    """Read and clear the error word of the cache operators on the current device (waits for the
    device): SV_ERR_WAIT where an attention gave up a wait and wrote NaN."""
    w = ctypes.c_uint32()
    _check(lib().spec_verify_cache_last_error(ctypes.byref(w)), "spec_verify_cache_last_error")
    return w.value


def spec_verify_reserve_host_io(ctx) -> None:
    _check(lib().spec_verify_reserve_host_io(ctx), "spec_verify_reserve_host_io")


def spec_verify_last_error(ctx) -> int:
    w = ctypes.c_uint32()
    _check(lib().spec_verify_last_error(ctx, ctypes.byref(w)), "spec_verify_last_error")
    return w.value


def spec_verify_set_profiling(ctx, enable: bool) -> None:
    _check(lib().spec_verify_set_profiling(ctx, int(enable)), "spec_verify_set_profiling")


def spec_verify_get_profile(ctx):
    ms = (ctypes.c_double * len(KERNELS))()
    calls = ctypes.c_int64()
    _check(lib().spec_verify_get_profile(ctx, ms, ctypes.byref(calls)), "spec_verify_get_profile")
    return dict(zip(KERNELS, list(ms))), calls.value


def spec_verify_set_chunks(ctx, stats_chunk: int = 0) -> None:
    _check(lib().spec_verify_set_chunks(ctx, stats_chunk), "spec_verify_set_chunks")


def spec_verify_launches_per_run() -> int:
    return lib().spec_verify_launches_per_run()


def spec_verify_free(ctx) -> None:
    if ctx:
        lib().spec_verify_free(ctx)


def spec_verify_status_string(status: int) -> str:
    return _status_string(status)


# ---- row operators -------------------------------------------------------------------------

def _row_matrix(name, t, dtypes, shape, device):
    """A 2-d device tensor whose rows are contiguous (any row stride), checked."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    rows, cols = shape
    if (cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < cols):
        raise ValueError(f"{name}'s rows must be contiguous and must not overlap")
    return t.data_ptr(), (t.stride(0) if rows > 1 else cols)


def _row_array(name, t, dtype, shape, device):
    """Address of a contiguous device tensor of this shape (None stays None), checked."""
    if t is None:
        return None
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be contiguous")


def _rows_of(logits):
    """(dtype code, rows, vocabulary, address, stride) of the logits of a row operator."""
    import torch

    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab_size]")
    if not logits.is_cuda:
        raise ValueError("logits must be on a CUDA device")
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"unsupported logits dtype {logits.dtype}")
    rows, vocab = logits.shape
    ptr, stride = _row_matrix("logits", logits, (logits.dtype,), (rows, vocab), logits.device)
    return SV_BF16 if logits.dtype == torch.bfloat16 else SV_F32, rows, vocab, ptr, stride


def _current_stream(index: int) -> int:
    """Handle of the current stream of device `index` (without making a stream object, which costs
    a fifth of a small call)."""
    import torch

    return torch._C._cuda_getCurrentRawStream(index)


def _row_outputs(out, want, device, stream):
    """The output tensors (name, dtype, shape): those given, one for each, or new ones, of the
    memory that belongs to the stream that writes them."""
    import torch

    if out is None:
        if stream is not None and _stream_handle(stream) != _current_stream(device.index):
            with torch.cuda.stream(torch.cuda.ExternalStream(_stream_handle(stream), device)):
                return _row_outputs(None, want, device, None)
        return [torch.empty(shape, dtype=dtype, device=device) for _, dtype, shape in want]
    if len(out) != len(want):
        raise ValueError("out must hold " + ", ".join(name for name, _, _ in want))
    return list(out)


def sample(logits, uniforms, temperature=None, *, top_k=None, top_p=None, min_p=None,
           logprob: bool = False, probs: bool = False, out=None, stream=None):
    """Draw one token of every row of logits ([rows, vocab_size] bfloat16 or float32, rows
    contiguous) by the given uniform numbers ([rows] float32 in [0, 1)): softmax at the
    temperature, of the tokens that top_k ([rows] int32), top_p and min_p ([rows] float32) keep,
    each None for no such constraint; the exact rules stand at spec_verify_sample in
    include/spec_verify.h. Temperature 0 or top_k 1 takes the largest logit.

    Returns (tokens int32 [rows]), with logprob=True also the tokens' log-probabilities, and with
    probs=True also the distributions they were drawn from, [rows, vocab_size] float32, which
    SpecVerify.run takes as draft_probs. out: tensors to write instead of new ones, in that
    order (the distributions' rows may be further apart than vocab_size). Runs on the logits'
    device, on `stream` or that device's current stream; no scratch memory, so calls may overlap.
    """
    import torch

    dtype, rows, vocab, ptr, stride = _rows_of(logits)
    dev = logits.device
    f32, i32 = torch.float32, torch.int32
    want = [("tokens", i32, (rows,))]
    if logprob:
        want.append(("logprob", f32, (rows,)))
    if probs:
        want.append(("probs", f32, (rows, vocab)))
    got = _row_outputs(out, want, dev, stream)
    pp, pstride = _row_matrix("probs", got[-1], (f32,), (rows, vocab), dev) if probs else (None, 0)
    args = SampleArgs(ptr, stride, _row_array("temperature", temperature, f32, (rows,), dev),
                      _row_array("top_k", top_k, i32, (rows,), dev),
                      _row_array("top_p", top_p, f32, (rows,), dev),
                      _row_array("min_p", min_p, f32, (rows,), dev),
                      _row_array("uniforms", uniforms, f32, (rows,), dev),
                      _row_array("tokens", got[0], i32, (rows,), dev),
                      _row_array("logprob", got[1], f32, (rows,), dev) if logprob else None,
                      pp, pstride, rows, vocab, dtype, dev.index)
    spec_verify_sample(args, _current_stream(dev.index) if stream is None else stream)
    return tuple(got)


def logprobs(logits, tokens=None, *, num_top: int = 0, temperature=None, cu_num_draft=None,
             out=None, stream=None):
    """Log-probabilities over the whole vocabulary of rows of logits ([rows, vocab_size] bfloat16
    or float32, rows contiguous), at temperature 1 or the given one ([rows] float32).

    tokens: [rows] int32, or with cu_num_draft ([num_reqs + 1] int32) the `sampled`
    [num_reqs, max_spec_len + 1] of a verification whose target logits these are. Returns
    (log-probability float32, rank int32: 1 + the number of larger logits), both [rows], and with
    num_top also the best tokens and their log-probabilities, [rows, num_top]; only these two
    where tokens is None. A row whose token is outside the vocabulary (the -1 behind a request's
    last token) is left out: -inf, 0, -1, -inf. out: tensors to write instead of new ones, in that
    order. Runs on the logits' device, on `stream` or that device's current stream; no scratch
    memory, so calls may overlap."""
    import torch

    dtype, rows, vocab, ptr, stride = _rows_of(logits)
    dev = logits.device
    f32, i32 = torch.float32, torch.int32
    if not 0 <= num_top <= SV_MAX_TOP:
        raise ValueError(f"num_top must be in [0, {SV_MAX_TOP}]")
    if tokens is None and (num_top == 0 or cu_num_draft is not None):
        raise ValueError("without tokens, num_top best tokens of every row are all there is")
    want = [("logprob", f32, (rows,)), ("rank", i32, (rows,))] if tokens is not None else []
    if num_top:
        want += [("top_ids", i32, (rows, num_top)), ("top_logprobs", f32, (rows, num_top))]
    got = _row_outputs(out, want, dev, stream)
    at = [_row_array(name, t, d, shape, dev) for t, (name, d, shape) in zip(got, want)]
    if tokens is None:
        at = [None, None, *at]
    elif not num_top:
        at += [None, None]
    num_reqs = width = 0
    if cu_num_draft is not None:
        num_reqs = cu_num_draft.numel() - 1
        if (tokens.dim() != 2 or tokens.shape[0] != num_reqs or (num_reqs == 0 and rows)
                or tokens.shape[1] < 1):
            raise ValueError("with cu_num_draft, tokens must be [num_reqs, max_spec_len + 1]")
        width = tokens.shape[1]
    args = LogprobsArgs(ptr, stride, _row_array("temperature", temperature, f32, (rows,), dev),
                        _row_array("tokens", tokens, i32, (num_reqs, width) if width else (rows,), dev),
                        _row_array("cu_num_draft", cu_num_draft, i32, (num_reqs + 1,), dev),
                        *at, width, num_reqs, num_top, rows, vocab, dtype, dev.index)
    spec_verify_logprobs(args, _current_stream(dev.index) if stream is None else stream)
    return tuple(got)


# ---- cache operators -----------------------------------------------------------------------

_CODES = {}   # element types of the cache operators and their codes
_torch = None  # what the cache operators take of PyTorch, looked up once: a call's lookups are a good part of its time


class _Torch:
    """PyTorch's types and functions that a call of a cache operator uses, and the library's functions."""

    def __init__(self):
        import torch

        self.int32, self.float32, self.uint8, self.e4m3 = torch.int32, torch.float32, torch.uint8, torch.float8_e4m3fn
        self.empty, self.stream = torch.empty, torch._C._cuda_getCurrentRawStream
        _CODES.update({torch.bfloat16: SV_BF16, torch.float16: SV_F16, torch.float8_e4m3fn: SV_E4M3})
        self.append, self.attention, self.byref = lib().spec_verify_cache_append, lib().spec_verify_cache_attention, ctypes.byref


def _cache_torch():
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _rows_code(name, t) -> int:
    """Type code of a [rows, heads, head_dim] tensor of the rows, checked."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows, {name}_heads, head_dim]" if name == "q" else f"{name} must be [rows, kv_heads, head_dim]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    code = _CODES.get(t.dtype)
    if code is None or code == SV_E4M3:
        raise ValueError(f"{name} has the unsupported dtype {t.dtype}")
    return code


def _head_rows(name, t, shape, dtype, index):
    """(address, row stride, head stride) of a [rows, heads, head_dim] tensor on device `index` whose heads
    are contiguous, checked."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == index:
        row, head, one = t.stride()
        at = t.data_ptr()
        if not (one != 1 or at & 15 or (row & 7 and shape[0] != 1) or (head & 7 and shape[1] != 1)):
            return at, row, head
        raise ValueError(f"{name}'s heads must be contiguous, its address and strides multiples of 16 bytes")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _whole(name, t, dtype, shape, index):
    """Address of a contiguous tensor of this shape on device `index`, checked."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    raise ValueError(f"{name} must be contiguous")


def _step_of(T, k_cache, v_cache, page_table, lengths, cu_num_draft, k_scale, v_scale, rows, heads, dim, dtype,
             index):
    """The arguments that the cache operators share, checked: (strides of the caches, the page table and what
    follows it, the scales, sizes of the pool, heads, type code, number of requests)."""
    shape, kind = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or shape[3] != dim or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [pages, page_size, kv_heads, head_dim], head_dim that of the rows")
    if v_cache.dtype is not kind or (kind is not dtype and kind is not T.e4m3):
        raise ValueError(f"caches have dtype {kind} and {v_cache.dtype}, expected {dtype} or torch.float8_e4m3fn")
    if k_cache.get_device() != index or v_cache.get_device() != index:
        raise ValueError(f"caches are on {k_cache.device} and {v_cache.device}, expected cuda:{index}")
    k_page, k_slot, k_head, k_one = k_cache.stride()
    v_page, v_slot, v_head, v_one = v_cache.stride()
    if k_one != 1 or v_one != 1:
        raise ValueError("the caches' heads must be contiguous")
    pages, page, hk, _ = shape
    if heads is not None and hk != heads:
        raise ValueError(f"the caches hold {hk} heads, the rows {heads}")
    n = lengths.numel()
    if page_table.dim() != 2 or lengths.dim() != 1 or page_table.shape[0] != n:
        raise ValueError("page_table must be [num_reqs, pages], lengths [num_reqs]")
    width = page_table.shape[1]
    if page_table.dtype is not T.int32 or page_table.get_device() != index:
        raise ValueError(f"page_table must be int32 on cuda:{index}")
    if (pages | page | width | n | rows) >> 31:  # (the library's are 32 bits)
        raise ValueError("pages, page_size, requests and rows must be below 2^31")
    table_stride, one = page_table.stride()
    if n <= 1:
        table_stride = width
    if (width > 1 and one != 1) or table_stride < width:
        raise ValueError("page_table's rows must be contiguous and must not overlap")
    cu = ks = vs = None
    if cu_num_draft is not None:
        cu = _whole("cu_num_draft", cu_num_draft, T.int32, (n + 1,), index)
    elif rows < n:
        raise ValueError(f"without cu_num_draft every request has a row: {n} requests, {rows} rows")
    code = _CODES[kind]
    if k_scale is not None or v_scale is not None:
        if code != SV_E4M3:
            raise ValueError("scales belong to float8_e4m3fn caches")
        ks = None if k_scale is None else _whole("k_scale", k_scale, T.float32, (hk,), index)
        vs = None if v_scale is None else _whole("v_scale", v_scale, T.float32, (hk,), index)
    return ((k_page, k_slot, k_head, v_page, v_slot, v_head),
            (page_table.data_ptr(), table_stride, _whole("lengths", lengths, T.int32, (n,), index), cu),
            (ks, vs), (pages, page, width), hk, code, n)


def _new(T, shape, dtype, device, stream):
    """A new tensor, of the memory that belongs to the stream that works on it."""
    if stream is None:
        return T.empty(shape, dtype=dtype, device=device)
    return _row_outputs(None, [("", dtype, shape)], device, stream)[0]


def cache_append(k, v, k_cache, v_cache, page_table, lengths, *, q=None, inv_freq=None, cu_num_draft=None,
                 positions=None, axes=None, interleaved: bool = False, k_scale=None, v_scale=None, out=None,
                 stream=None):
    """Append the keys and values of a step's rows to the paged cache, the keys turned by their
    positions, and turn the queries.

    k, v: [rows, kv_heads, head_dim] bfloat16 or float16 (views of one projection, say); row
    cu_num_draft[i] + i + j is the j-th new token of request i (cu_num_draft [num_reqs + 1] int32, the
    verification's; None: one row a request) at place lengths[i] + j ([num_reqs] int32, the tokens cached
    before; negative: the request takes no part). k_cache, v_cache: [pages, page_size, kv_heads, head_dim]
    in any layout whose heads are contiguous, of the rows' dtype, or float8_e4m3fn with k_scale and v_scale
    ([kv_heads] float32: what is stored is the value divided by its head's scale) or without. page_table:
    [num_reqs, pages_of_a_request] int32.

    inv_freq ([rotary_dim / 2] float32, None: nothing is turned): the rotation of the first rotary_dim
    elements of q's and k's heads, pair m by the angle position * inv_freq[m]; pairs are half of rotary_dim
    apart, or neighbours with interleaved=True. The position is the row's place, or with positions
    ([num_axes, rows] int32, or [rows]) that of axis axes[m] (a sequence of rotary_dim / 2 axis numbers;
    None: axis 0).

    Returns the turned queries [rows, q_heads, head_dim] (None without q): a new tensor, or `out`, which
    may be q itself. Runs on k's device, on `stream` or that device's current stream. The exact rules stand
    at spec_verify_cache_append in include/spec_verify.h."""
    T = _torch or _cache_torch()
    code = _rows_code("k", k)
    shape, dtype, index = k.shape, k.dtype, k.get_device()
    rows, hk, dim = shape
    strides, step, scales, pool, _, cache_code, n = _step_of(T, k_cache, v_cache, page_table, lengths, cu_num_draft,
                                                             k_scale, v_scale, rows, hk, dim, dtype, index)
    k_at, k_row, k_head = _head_rows("k", k, shape, dtype, index)
    v_at, v_row, v_head = _head_rows("v", v, shape, dtype, index)
    qp = op = (None, 0, 0)
    hq = half = num_axes = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [rows, q_heads, head_dim]")
        hq = q.shape[1]
        qp = _head_rows("q", q, (rows, hq, dim), dtype, index)
        if out is None:
            out = _new(T, (rows, hq, dim), dtype, k.device, stream)
        op = qp if out is q else _head_rows("out", out, (rows, hq, dim), dtype, index)
    elif out is not None:
        raise ValueError("out without q")
    inv = pos = axis_bytes = None
    if inv_freq is not None:
        half = inv_freq.numel()
        inv = _whole("inv_freq", inv_freq, T.float32, (half,), index)
    if positions is not None:
        if positions.dim() == 1:
            positions = positions[None]
        num_axes = positions.shape[0]
        pos = _whole("positions", positions, T.int32, (num_axes, rows), index)
    if axes is not None:
        if len(axes) != half:
            raise ValueError(f"axes must name the axis of each of the {half} pairs")
        try:
            axis_bytes = bytes(list(axes))  # (its numbers: bytes of an array are the array's memory)
        except TypeError as e:
            raise ValueError("axes must be whole numbers") from e
    args = CacheAppendArgs(qp[0], k_at, v_at, op[0], k_cache.data_ptr(), v_cache.data_ptr(), qp[1], qp[2], k_row, k_head,
                           v_row, v_head, op[1], op[2], *strides, *step, pos, rows, inv, *scales, axis_bytes, rows, n, hq,
                           hk, dim, 2 * half, 1 if interleaved else 0, num_axes, *pool, code, cache_code, index)
    status = T.append(T.byref(args), T.stream(index) if stream is None else _stream_handle(stream))
    if status:
        _check(status, "spec_verify_cache_append")
    return out


def cache_attention(q, k_cache, v_cache, page_table, lengths, *, cu_num_draft=None, scale=None, window: int = 0,
                    k_scale=None, v_scale=None, lse: bool = False, out=None, stream=None):
    """Attention of a step's rows over the paged cache: q [rows, q_heads, head_dim] (bfloat16 or float16,
    head_dim 64, 128 or 256), laid out as for :func:`cache_append`, which has appended the rows' own keys
    under the same page_table, lengths and cu_num_draft. The row at place x = lengths[i] + j sees the keys at
    places 0 to x of its request, with window > 0 the last `window` of them; query head g reads key head
    g // (q_heads // kv_heads). scale: the factor of q . k, head_dim ** -0.5 by default. A row that sees no key
    (a request of negative length) gets 0.

    Returns (out [rows, q_heads, head_dim] of q's dtype,), with lse=True also the logarithm of the sum of
    exponentials, [rows, q_heads] float32 (-inf where no key is seen), with which parts of an attention can be
    joined. out: tensors to write instead of new ones, in that order. Rows behind the last request's are left
    as they are. Runs on q's device, on `stream` or that device's current stream; the workspace is the call's own, so
    calls may overlap. Should the device lose a copy, rows get NaN and spec_verify_cache_last_error() is not 0. The exact
    rules stand at spec_verify_cache_attention in include/spec_verify.h."""
    T = _torch or _cache_torch()
    code = _rows_code("q", q)
    shape, dtype, index = q.shape, q.dtype, q.get_device()
    rows, hq, dim = shape
    strides, step, scales, pool, hk, cache_code, n = _step_of(T, k_cache, v_cache, page_table, lengths, cu_num_draft,
                                                              k_scale, v_scale, rows, None, dim, dtype, index)
    if hk < 1 or hq < 1 or hq % hk:
        raise ValueError(f"{hq} query heads are not a multiple of the caches' {hk} heads")
    if window >> 31:
        raise ValueError("window must be within 0 and 2^31 - 1")
    q_at, q_row, q_head = _head_rows("q", q, shape, dtype, index)
    device = q.device
    if out is None:
        out = [_new(T, shape, dtype, device, stream)]
        if lse:
            out.append(_new(T, (rows, hq), T.float32, device, stream))
    elif len(out) != 1 + bool(lse):
        raise ValueError("out must hold out, lse" if lse else "out must hold out")
    o_at, o_row, o_head = _head_rows("out", out[0], shape, dtype, index)
    l_at = _whole("lse", out[1], T.float32, (rows, hq), index) if lse else None
    space = _new(T, SV_CACHE_WORKSPACE, T.uint8, device, stream)
    args = CacheAttentionArgs(q_at, k_cache.data_ptr(), v_cache.data_ptr(), o_at, l_at, q_row, q_head, o_row, o_head,
                              *strides, *step, *scales, space.data_ptr(), SV_CACHE_WORKSPACE,
                              dim ** -0.5 if scale is None else scale, window, rows, n, hq, hk, dim, *pool, code,
                              cache_code, index)
    status = T.attention(T.byref(args), T.stream(index) if stream is None else _stream_handle(stream))
    if status:
        _check(status, "spec_verify_cache_attention")
    return tuple(out)


# ---- convenience owner ---------------------------------------------------------------------

def _dtype_code(logits_dtype) -> int:
    s = str(logits_dtype).lower()
    if "bf16" in s or "bfloat16" in s:
        return SV_BF16
    if "f32" in s or "float32" in s or s in ("float", "torch.float"):
        return SV_F32
    raise ValueError(f"unsupported logits dtype {logits_dtype}")


class SpecVerify:
    """Owns one context. Tensors passed to :meth:`run` must live on the context's device."""

    def __init__(self, max_num_reqs: int, max_spec_len: int, vocab_size: int, logits_dtype="bf16",
                 has_draft_probs: bool = True, device: int = 0, *, draft_logits: bool = False):
        self.max_num_reqs, self.max_spec_len, self.vocab_size = max_num_reqs, max_spec_len, vocab_size
        self.dtype_code = _dtype_code(logits_dtype)
        self.device = device
        draft_input = (SV_DRAFT_PROBS if has_draft_probs else 0) | (SV_DRAFT_LOGITS if draft_logits else 0)
        self.ctx = spec_verify_init(max_num_reqs, max_spec_len, vocab_size, self.dtype_code,
                                    draft_input, device)

    def run(self, logits, draft_ids, draft_probs, cu_num_draft, temperature, is_greedy, seed: int,
            *, req_index_base: int = 0, max_spec_len: int | None = None, out=None,
            row_stats: bool = False, stream=None, draft_logits=None, partial_prefill=None,
            frequency_penalty=None, output_bin_counts=None, counts_row=None, top_k=None,
            top_p=None, stats_out=None, fp64_gumbel: bool = False):
        """Verify a batch held in device tensors. Returns (sampled, num_sampled, num_rejected)
        and, with row_stats=True, also (row_max, row_sumexp, row_argmax).

        draft_logits ([num_draft_tokens, vocab_size], the logits' dtype) replaces draft_probs:
        q is then computed inside the call (context created with draft_logits=True).
        partial_prefill ([num_reqs] uint8): requests still in a chunked prefill, which report
        no token. frequency_penalty ([num_reqs] float32) with output_bin_counts ([rows, V]
        int32) and counts_row ([num_reqs] int32, optional): the frequency penalty. top_k
        ([num_reqs] int32), top_p ([num_reqs] float32): sampling constraints. Any of these
        goes through spec_verify_run_batch. out / stats_out: caller-provided output tensors
        (sampled, num_sampled, num_rejected) / (row_max, row_sumexp, row_argmax).
        fp64_gumbel=True draws the race noise in binary64 (the fp64 Gumbel option)."""
        import torch
        num_reqs = cu_num_draft.numel() - 1
        nd = draft_ids.numel()
        kmax = self.max_spec_len if max_spec_len is None else max_spec_len
        if logits.dim() != 2 or logits.shape[0] != nd + num_reqs or logits.shape[1] != self.vocab_size:
            raise ValueError("logits must be [num_draft_tokens + num_reqs, vocab_size]")
        if draft_logits is not None:
            if draft_probs is not None:
                raise ValueError("give draft_probs or draft_logits, not both")
            if (draft_logits.dim() != 2 or draft_logits.shape[0] != nd
                    or draft_logits.shape[1] != self.vocab_size or draft_logits.dtype != logits.dtype):
                raise ValueError("draft_logits must be [num_draft_tokens, vocab_size] of the logits' dtype")
        dev = logits.device
        if out is None:
            out = (torch.empty((num_reqs, kmax + 1), dtype=torch.int32, device=dev),
                   torch.empty(num_reqs, dtype=torch.int32, device=dev),
                   torch.empty(num_reqs, dtype=torch.int32, device=dev))
        stats = (None, None, None)
        if row_stats and stats_out is not None:
            stats = tuple(stats_out)
        elif row_stats:
            R = nd + num_reqs
            stats = (torch.empty(R, dtype=torch.float32, device=dev),
                     torch.empty(R, dtype=torch.float32, device=dev),
                     torch.empty(R, dtype=torch.int32, device=dev))
        extras = (partial_prefill, frequency_penalty, output_bin_counts, counts_row, top_k, top_p)
        if any(x is not None for x in extras) or fp64_gumbel:
            if output_bin_counts is not None and (output_bin_counts.dim() != 2
                                                  or output_bin_counts.shape[1] != self.vocab_size):
                raise ValueError("output_bin_counts must be [rows, vocab_size]")
            b = Batch(_ptr(logits), _ptr(draft_ids), _ptr(draft_probs), _ptr(draft_logits),
                      _ptr(cu_num_draft), _ptr(temperature), _ptr(is_greedy),
                      _ptr(partial_prefill), _ptr(frequency_penalty), _ptr(output_bin_counts),
                      _ptr(counts_row), _ptr(top_k), _ptr(top_p), seed, req_index_base,
                      num_reqs, nd, kmax,
                      output_bin_counts.shape[0] if output_bin_counts is not None else 0,
                      int(bool(fp64_gumbel)))
            o = Outputs(*(_ptr(t) for t in (*out, *stats)))
            spec_verify_run_batch(self.ctx, b, o, cuda_stream=stream)
        elif draft_logits is not None:
            spec_verify_run_draft_logits(self.ctx, logits, draft_ids, draft_logits, cu_num_draft,
                                         temperature, is_greedy, seed, req_index_base, num_reqs,
                                         nd, kmax, *out, *stats, cuda_stream=stream)
        else:
            spec_verify_run(self.ctx, logits, draft_ids, draft_probs, cu_num_draft, temperature,
                            is_greedy, seed, req_index_base, num_reqs, nd, kmax, *out, *stats,
                            cuda_stream=stream)
        return (*out, *stats) if row_stats else out

    def reserve_host_io(self) -> None:
        spec_verify_reserve_host_io(self.ctx)

    def run_host(self, logits, draft_ids, draft_probs, cu_num_draft, temperature, is_greedy,
                 seed: int, sampled, num_sampled, num_rejected, *, req_index_base: int = 0,
                 max_spec_len: int | None = None, stream=None) -> None:
        """Verify a batch held in host memory (numpy arrays or CPU tensors; pinned memory
        gives asynchronous copies, and pinned draft_probs is read in place by the kernels);
        outputs are written to the host arrays given."""
        num_reqs = len(cu_num_draft) - 1
        nd = len(draft_ids)
        kmax = self.max_spec_len if max_spec_len is None else max_spec_len
        spec_verify_run_host(self.ctx, logits, draft_ids, draft_probs, cu_num_draft, temperature,
                             is_greedy, seed, req_index_base, num_reqs, nd, kmax, sampled,
                             num_sampled, num_rejected, cuda_stream=stream)

    def last_error(self) -> int:
        return spec_verify_last_error(self.ctx)

    def set_profiling(self, enable: bool) -> None:
        spec_verify_set_profiling(self.ctx, enable)

    def get_profile(self):
        return spec_verify_get_profile(self.ctx)

    def set_synthetic(self, rates) -> None:
        """Synthetic acceptance with these unconditional per-position rates ([] = off)."""
        spec_verify_set_synthetic(self.ctx, rates)

    def set_synthetic_length(self, mean_length: float, num_spec: int | None = None) -> None:
        """Synthetic acceptance with the minimum-variance rates of a target mean length."""
        n = self.max_spec_len if num_spec is None else num_spec
        spec_verify_set_synthetic(self.ctx, spec_verify_synthetic_rates(mean_length, n))

    def set_chunks(self, stats_chunk: int = 0) -> None:
        spec_verify_set_chunks(self.ctx, stats_chunk)

    def close(self) -> None:
        if self.ctx:
            spec_verify_free(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass
