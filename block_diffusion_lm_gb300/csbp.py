"""ctypes binding of libcsbp (include/csbp.h, csbp_vocab_ce.h,
csbp_generate.h): argument marshalling only.

Every step of the attention path runs in the library's kernels; PyTorch is
used here only to own device memory and to name the current CUDA stream.
There is no fallback: if libcsbp.so is missing or fails to load, every call
raises.
"""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcsbp.so")
INCLUDE = os.path.join(os.path.dirname(_PKG), "include")
HEADER = os.path.join(INCLUDE, "csbp.h")

OK = 0
STATUS = {0: "CSBP_OK", -1: "CSBP_ERR_INVALID", -2: "CSBP_ERR_UNSUPPORTED",
          -3: "CSBP_ERR_WORKSPACE", -4: "CSBP_ERR_CUDA", -5: "CSBP_ERR_TIMEOUT",
          -6: "CSBP_ERR_CAPACITY", -7: "CSBP_ERR_DEVICE"}


class CsbpError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")


class Problem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("L", ctypes.c_int32), ("M", ctypes.c_int32),
                ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("P", ctypes.c_int32), ("tile_q", ctypes.c_int32), ("tile_kv", ctypes.c_int32),
                ("has_clean_queries", ctypes.c_int32), ("scale", ctypes.c_float),
                ("window", ctypes.c_int32), ("clean_causal", ctypes.c_int32),
                ("bwd_chunk", ctypes.c_int32), ("per_rank", ctypes.c_int32),
                ("rank", ctypes.c_int32)]


class Inputs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("q_clean", "k_clean", "v_clean", "q_corr", "k_corr", "v_corr")] + [
                    ("stride_tok", ctypes.c_int64 * 6), ("stride_batch", ctypes.c_int64 * 6)]


class CeProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("d_model", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("chunk_rows", ctypes.c_int32), ("head_grad", ctypes.c_int32),
                ("grad_scale", ctypes.c_float)]


class ScheduleInfo(ctypes.Structure):
    _fields_ = [("n_fwd_tasks", ctypes.c_int32), ("n_fwd_segments", ctypes.c_int32),
                ("n_bwd_tasks", ctypes.c_int32), ("n_bwd_segments", ctypes.c_int32),
                ("tile_pairs", ctypes.c_int64), ("bytes", ctypes.c_int64),
                ("problem_key", ctypes.c_uint64)]


class KvCache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class CacheRows(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("table_pages", ctypes.c_int32), ("table", ctypes.c_void_p),
                ("start", ctypes.c_void_p), ("count", ctypes.c_void_p),
                ("stride_tok", ctypes.c_int64 * 2), ("stride_batch", ctypes.c_int64 * 2)]


class RotaryStruct(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("turns", ctypes.c_void_p)]


class AppendQueries(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int32), ("clear", ctypes.c_int32), ("q", ctypes.c_void_p),
                ("out", ctypes.c_void_p),
                ("stride_tok", ctypes.c_int64 * 2), ("stride_batch", ctypes.c_int64 * 2)]


class PagedProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "queries", "table_pages", "Hq", "causal", "window", "sinks")] + [
                    ("scale", ctypes.c_float)]


class PagedInputs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("stride_tok", ctypes.c_int64),
                ("stride_batch", ctypes.c_int64), ("table", ctypes.c_void_p),
                ("length", ctypes.c_void_p)]


class PrefixProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "queries", "prefix_len", "own_max", "Hq", "Hkv", "d", "causal")] + [
                    ("scale", ctypes.c_float)]


class PrefixInputs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("q", "k_prefix", "v_prefix", "k_own", "v_own", "own_len")] + [
                    ("stride_tok", ctypes.c_int64 * 5), ("stride_batch", ctypes.c_int64 * 5)]


class VerifyProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("drafts", ctypes.c_int32),
                ("vocab", ctypes.c_int32)] + [
                    (n, ctypes.c_int64) for n in ("p_row", "p_batch", "q_row", "q_batch")]


_lib = None
_lib_path = LIB_PATH
DEBUG_LIB_PATH = os.path.join(_PKG, "libcsbp_debug.so")


def use_library(path: str = LIB_PATH) -> None:
    """Bind later calls to the library at `path` (e.g. the debug build,
    DEBUG_LIB_PATH, whose kernels check their work-list records)."""
    global _lib, _lib_path
    _lib, _lib_path = None, path


def lib():
    """Load the bound library, libcsbp.so by default (raises if it was not
    built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_lib_path):
            raise RuntimeError(f"{_lib_path} not built: run block_diffusion_lm_gb300.build.build()")
        L = ctypes.CDLL(_lib_path)
        P = ctypes.POINTER
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.csbp_block_schedule.argtypes = [P(Problem), P(i32), P(i32), vp, i64, P(ScheduleInfo)]
        L.csbp_workspace_bytes.argtypes = [P(Problem), ctypes.c_int]
        L.csbp_workspace_bytes.restype = sz
        L.csbp_attn_fwd.argtypes = [P(Problem), P(Inputs), vp, P(ScheduleInfo), vp, vp, vp, vp,
                                    sz, vp]
        L.csbp_attn_bwd.argtypes = [P(Problem), P(Inputs), vp, P(ScheduleInfo), vp, vp, vp, vp,
                                    vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.csbp_attn_bwd_noalloc.argtypes = [P(Problem), P(Inputs), vp, P(ScheduleInfo), vp, vp,
                                            vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.csbp_attn_bwd_noalloc.restype = ctypes.c_int
        L.csbp_e4m3_to_bf16.argtypes = [vp, ctypes.c_float, vp, i64, vp]
        L.csbp_e4m3_to_bf16.restype = ctypes.c_int
        L.csbp_attn_bwd_noalloc_status.argtypes = [vp]
        L.csbp_attn_bwd_noalloc_status.restype = ctypes.c_int
        L.csbp_lse_merge.argtypes = [i32, P(vp), P(vp), i64, i32, i32, vp, vp, vp]
        L.csbp_check_status.argtypes = [vp, vp]
        L.csbp_status_string.argtypes = [ctypes.c_int]
        L.csbp_status_string.restype = ctypes.c_char_p
        L.csbp_version.restype = i32
        L.csbp_kernel_timing.argtypes = [i32]
        L.csbp_kernel_timing_read.argtypes = [P(ctypes.c_double), P(i32), P(ctypes.c_double),
                                              P(i32)]
        L.csbp_kernel_timing_read_kind.argtypes = [i32, P(ctypes.c_double), P(i32)]
        L.csbp_wait_selftest.argtypes = [i64, vp, vp]
        L.csbp_ce_workspace_bytes.argtypes = [P(CeProblem)]
        L.csbp_ce_workspace_bytes.restype = sz
        L.csbp_vocab_ce.argtypes = [P(CeProblem), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.csbp_cache_write.argtypes = [P(KvCache), P(CacheRows), vp, vp, vp]
        L.csbp_cache_read.argtypes = [P(KvCache), P(CacheRows), vp, vp, vp]
        L.csbp_rotary_turns.argtypes = [P(ctypes.c_double), i32, P(ctypes.c_uint64)]
        L.csbp_cache_append.argtypes = [P(KvCache), P(CacheRows), P(RotaryStruct), vp, vp,
                                        P(AppendQueries), vp]
        L.csbp_paged_workspace_bytes.argtypes = [P(PagedProblem), P(KvCache)]
        L.csbp_paged_workspace_bytes.restype = sz
        L.csbp_attn_paged.argtypes = [P(PagedProblem), P(KvCache), P(PagedInputs), vp, vp, vp,
                                      sz, vp]
        L.csbp_prefix_workspace_bytes.argtypes = [P(PrefixProblem)]
        L.csbp_prefix_workspace_bytes.restype = sz
        L.csbp_attn_prefix.argtypes = [P(PrefixProblem), P(PrefixInputs), vp, vp, vp, sz, vp]
        L.csbp_draft_verify.argtypes = [P(VerifyProblem)] + [vp] * 9
        for fn in ("csbp_cache_write", "csbp_cache_read", "csbp_rotary_turns",
                   "csbp_cache_append", "csbp_attn_paged", "csbp_attn_prefix",
                   "csbp_draft_verify", "csbp_block_schedule", "csbp_attn_fwd", "csbp_attn_bwd", "csbp_lse_merge",
                   "csbp_check_status", "csbp_kernel_timing", "csbp_kernel_timing_read",
                   "csbp_kernel_timing_read_kind", "csbp_vocab_ce", "csbp_wait_selftest"):
            getattr(L, fn).restype = ctypes.c_int
        _lib = L
    return _lib


def header_functions():
    """Names of the functions the headers under include/ declare."""
    names = set()
    for h in sorted(os.listdir(INCLUDE)):
        if h.endswith(".h"):
            with open(os.path.join(INCLUDE, h)) as f:
                text = f.read()
            names.update(re.findall(r"^\s*(?:const\s+)?[\w]+\s*\*?\s*(csbp_\w+)\s*\(", text, re.M))
    return sorted(names)


def _check(fn, status):
    if status != OK:
        raise CsbpError(fn, status)


def make_problem(batch, L, M, Hq, Hkv, d, P=1, has_clean_queries=True, scale=None,
                 tile=128, window=0, clean_causal=False, bwd_chunk=0, rank=None) -> Problem:
    """rank=None: every query row; rank=r: only the rows CSBP rank r of P owns."""
    return Problem(batch, L, M, Hq, Hkv, d, P, tile, tile, 1 if has_clean_queries else 0,
                   float(scale if scale is not None else d ** -0.5), int(window),
                   1 if clean_causal else 0, int(bwd_chunk), 0 if rank is None else 1,
                   0 if rank is None else int(rank))


def block_schedule(problem: Problem):
    """Host work list: returns (block_owner, chunk_owner, words[int32], info)."""
    info = ScheduleInfo()
    B = problem.L // problem.M if problem.M > 0 else 0
    bo = np.zeros(max(B, 1), np.int32)
    co = np.zeros(max(2 * problem.P, 1), np.int32)
    st = lib().csbp_block_schedule(ctypes.byref(problem),
                                   bo.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                   co.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                   None, 0, ctypes.byref(info))
    if st != -6:
        _check("csbp_block_schedule", st)
    words = np.zeros(info.bytes // 4, np.int32)
    st = lib().csbp_block_schedule(ctypes.byref(problem),
                                   bo.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                   co.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                   words.ctypes.data_as(ctypes.c_void_p), words.nbytes,
                                   ctypes.byref(info))
    _check("csbp_block_schedule", st)
    return bo[:B], co[:2 * problem.P], words, info


def kernel_timing(enable: bool) -> None:
    """Start (clearing the record) or stop event timing of the main kernels."""
    _check("csbp_kernel_timing", lib().csbp_kernel_timing(1 if enable else 0))


def kernel_timing_read():
    """(fwd_kernel_ms, n_fwd, bwd_kernel_ms, n_bwd) summed over the record."""
    fm, bm = ctypes.c_double(), ctypes.c_double()
    fn, bn = ctypes.c_int32(), ctypes.c_int32()
    _check("csbp_kernel_timing_read",
           lib().csbp_kernel_timing_read(ctypes.byref(fm), ctypes.byref(fn), ctypes.byref(bm),
                                         ctypes.byref(bn)))
    return fm.value, fn.value, bm.value, bn.value


def kernel_timing_read_kind(kind: int):
    """(ms, launches) of one timer kind: 0 fwd, 1 bwd, 2 CE logits GEMM,
    3 CE row kernel, 4 CE dH GEMM, 5 CE dW GEMM, 11 cache write and append, 12
    cache read, 13 prefix and paged attention, 14 the joining of their pieces in a
    kernel of its own, 15 draft verification."""
    ms, n = ctypes.c_double(), ctypes.c_int32()
    _check("csbp_kernel_timing_read_kind",
           lib().csbp_kernel_timing_read_kind(kind, ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


def workspace_bytes(problem: Problem, which: int) -> int:
    return int(lib().csbp_workspace_bytes(ctypes.byref(problem), which))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class _Checks:
    """Refuse tensors the library would misread: the C ABI sees only
    pointers, so dtype, shape and contiguity of every argument are checked
    first, then (in `done`) that all of them are on a CUDA device."""

    def __init__(self, fn):
        self.fn = fn
        self.seen = []

    def tensor(self, name, t, dtype, shape, required=True, strided=False):
        """`strided`: token and batch strides are free (the library takes
        them); heads and features must still be contiguous."""
        fn = self.fn
        if t is None:
            if required:
                raise ValueError(f"{fn}: {name} is required")
            return
        if t.dtype != dtype:
            raise ValueError(f"{fn}: {name} must be {dtype}, got {t.dtype}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{fn}: {name} must have shape {tuple(shape)}, "
                             f"got {tuple(t.shape)}")
        if strided:
            if t.stride(3) != 1 or (t.shape[2] > 1 and t.stride(2) != t.shape[3]):
                raise ValueError(f"{fn}: {name} must have contiguous heads and features "
                                 f"(strides [..., d, 1]), got {tuple(t.stride())}")
            # a zero stride means "contiguous" to the library, so a broadcast
            # (expanded) batch or token dimension would be misread
            if any(t.shape[i] > 1 and t.stride(i) == 0 for i in (0, 1)):
                raise ValueError(f"{fn}: {name} has a broadcast (stride-0) batch or token "
                                 f"dimension; materialise it first")
            row = t.shape[2] * t.shape[3]
            if t.shape[1] > 1 and (t.stride(1) < row or t.stride(1) % 8):
                raise ValueError(f"{fn}: {name} token stride {t.stride(1)} must be >= H*d = "
                                 f"{row} and a multiple of 8")
            if t.shape[0] > 1 and (t.stride(0) < t.shape[1] * max(t.stride(1), row)
                                   or t.stride(0) % 8):
                raise ValueError(f"{fn}: {name} batch entries must not interleave (batch "
                                 f"stride >= L x token stride, a multiple of 8); make a "
                                 f"sequence-first layout batch-first")
        elif not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must be contiguous")
        self.seen.append((name, t))

    def attn(self, problem, tensors):
        """q/o/dq/dO bf16 [batch][L][Hq][d], k/v/dk/dv bf16 [batch][L][Hkv][d],
        lse fp32 [batch][2][Hq][L]; clean-query tensors are optional when the
        problem has no clean queries."""
        import torch
        q = (problem.batch, problem.L, problem.Hq, problem.d)
        kv = (problem.batch, problem.L, problem.Hkv, problem.d)
        for name, t in tensors.items():
            if name == "lse":
                self.tensor(name, t, torch.float32, (problem.batch, 2, problem.Hq, problem.L))
                continue
            key_side = name.startswith(("k_", "v_", "dk_", "dv_"))
            optional = not key_side and name.endswith("_clean") and not problem.has_clean_queries
            self.tensor(name, t, torch.bfloat16, kv if key_side else q, required=not optional,
                        strided=name in _INPUT_NAMES)

    def done(self):
        for name, t in self.seen:
            if not t.is_cuda:
                raise ValueError(f"{self.fn}: {name} must be a CUDA tensor")


_INPUT_NAMES = ("q_clean", "k_clean", "v_clean", "q_corr", "k_corr", "v_corr")


def _inputs(inputs):
    """csbp_inputs from a dict of [batch][L][H][d] tensors: pointers, and the
    token / batch strides of each (0 where a dimension has one entry)."""
    ts = [inputs.get(n) for n in _INPUT_NAMES]
    tok = [0 if t is None or t.shape[1] == 1 else t.stride(1) for t in ts]
    bat = [0 if t is None or t.shape[0] == 1 else t.stride(0) for t in ts]
    return Inputs(*(_ptr(t) for t in ts), (ctypes.c_int64 * 6)(*tok),
                  (ctypes.c_int64 * 6)(*bat))


def _fresh(stream, make):
    """The tensors that make() allocates (and fills) for a call on `stream`, in a
    tuple or dict.  They come from the stream that the call runs on: on the
    current one, where that is another, a fill or an earlier user of the memory
    could still be waiting and land after the kernel.  The current stream, where
    the caller goes on, keeps them allocated until it has done with them too."""
    import torch
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        out = make()
    for t in out.values() if isinstance(out, dict) else out:
        if t is not None and t.is_cuda:
            t.record_stream(torch.cuda.current_stream(t.device))
    return out


def _zeros(shape, device):
    """Zeroed bytes that a handle keeps, ready for any stream: the host waits
    for the fill, once per handle.  (Under capture the fill is part of the graph.)"""
    import torch
    t = torch.zeros(shape, dtype=torch.uint8, device=device)
    if t.is_cuda:
        with torch.cuda.device(t.device):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()
    return t


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def attn_fwd(problem, inputs: dict, work_dev, info, o_clean, o_corr, lse, workspace, stream=None):
    import torch
    c = _Checks("csbp_attn_fwd")
    c.attn(problem, {**{n: inputs.get(n) for n in _INPUT_NAMES},
                     "o_clean": o_clean, "o_corr": o_corr, "lse": lse})
    c.tensor("work", work_dev, torch.int32, None)
    c.tensor("workspace", workspace, torch.uint8, None)
    c.done()
    inp = _inputs(inputs)
    st = lib().csbp_attn_fwd(ctypes.byref(problem), ctypes.byref(inp), _ptr(work_dev),
                             ctypes.byref(info), _ptr(o_clean), _ptr(o_corr), _ptr(lse),
                             _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _stream_ptr(stream))
    _check("csbp_attn_fwd", st)


def _check_bwd(c, problem, inputs, work_dev, o_clean, o_corr, lse, do_clean, do_corr, grads):
    import torch
    names = ("dq_clean", "dq_corr", "dk_clean", "dv_clean", "dk_corr", "dv_corr")
    c.attn(problem, {**{n: inputs.get(n) for n in _INPUT_NAMES},
                     "o_clean": o_clean, "o_corr": o_corr, "lse": lse,
                     "do_clean": do_clean, "do_corr": do_corr,
                     **{n: grads.get(n) for n in names}})
    c.tensor("work", work_dev, torch.int32, None)


def attn_bwd(problem, inputs: dict, work_dev, info, o_clean, o_corr, lse, do_clean, do_corr,
             grads: dict, workspace, stream=None):
    import torch
    c = _Checks("csbp_attn_bwd")
    _check_bwd(c, problem, inputs, work_dev, o_clean, o_corr, lse, do_clean, do_corr, grads)
    c.tensor("workspace", workspace, torch.uint8, None)
    c.done()
    inp = _inputs(inputs)
    st = lib().csbp_attn_bwd(ctypes.byref(problem), ctypes.byref(inp), _ptr(work_dev),
                             ctypes.byref(info), _ptr(o_clean), _ptr(o_corr), _ptr(lse),
                             _ptr(do_clean), _ptr(do_corr), _ptr(grads.get("dq_clean")),
                             _ptr(grads["dq_corr"]), _ptr(grads["dk_clean"]),
                             _ptr(grads["dv_clean"]), _ptr(grads["dk_corr"]),
                             _ptr(grads["dv_corr"]), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _check("csbp_attn_bwd", st)


def attn_bwd_noalloc(problem, inputs: dict, work_dev, info, o_clean, o_corr, lse, do_clean,
                     do_corr, grads: dict, stream=None):
    """csbp_attn_bwd_noalloc: the backward with the library's own fixed
    scratch instead of a caller workspace (for callers that cannot allocate
    device memory; calls on one device must not overlap)."""
    c = _Checks("csbp_attn_bwd_noalloc")
    _check_bwd(c, problem, inputs, work_dev, o_clean, o_corr, lse, do_clean, do_corr, grads)
    c.done()
    inp = _inputs(inputs)
    st = lib().csbp_attn_bwd_noalloc(ctypes.byref(problem), ctypes.byref(inp), _ptr(work_dev),
                                     ctypes.byref(info), _ptr(o_clean), _ptr(o_corr), _ptr(lse),
                                     _ptr(do_clean), _ptr(do_corr), _ptr(grads.get("dq_clean")),
                                     _ptr(grads["dq_corr"]), _ptr(grads["dk_clean"]),
                                     _ptr(grads["dv_clean"]), _ptr(grads["dk_corr"]),
                                     _ptr(grads["dv_corr"]), _stream_ptr(stream))
    _check("csbp_attn_bwd_noalloc", st)


def attn_bwd_noalloc_status(stream=None):
    """csbp_attn_bwd_noalloc_status: synchronise the stream and raise if a
    device wait of the last allocation-free backward gave up."""
    _check("csbp_attn_bwd_noalloc_status", lib().csbp_attn_bwd_noalloc_status(_stream_ptr(stream)))


def e4m3_to_bf16(x, scale: float, out=None, stream=None):
    """csbp_e4m3_to_bf16: decode fp8 E4M3 bytes (a torch uint8 or
    float8_e4m3fn CUDA tensor) times `scale` into bf16 (out: bf16 tensor of
    the same shape, allocated if None)."""
    import torch
    c = _Checks("csbp_e4m3_to_bf16")
    if x is None or x.dtype not in (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8)):
        raise ValueError("csbp_e4m3_to_bf16: x must be a uint8 or float8_e4m3fn tensor")
    if not x.is_contiguous():
        raise ValueError("csbp_e4m3_to_bf16: x must be contiguous")
    if out is None:
        out, = _fresh(stream, lambda: (
            torch.empty(x.shape, dtype=torch.bfloat16, device=x.device),))
    c.tensor("out", out, torch.bfloat16, tuple(x.shape))
    c.seen.append(("x", x))
    c.done()
    _check("csbp_e4m3_to_bf16", lib().csbp_e4m3_to_bf16(_ptr(x), float(scale), _ptr(out),
                                                        x.numel(), _stream_ptr(stream)))
    return out


def lse_merge(o_parts, lse_parts, o_out, lse_out, stream=None):
    """o_parts: list of fp32 [rows, Hq, d] device tensors; lse_parts: list of
    fp32 [Hq, rows]; o_out bf16 [rows, Hq, d]; lse_out fp32 [Hq, rows]."""
    import torch
    c = _Checks("csbp_lse_merge")
    n = len(o_parts)
    if n < 1 or len(lse_parts) != n:
        raise ValueError("csbp_lse_merge: needs one LSE part per output part, at least one")
    rows, Hq, d = o_parts[0].shape
    for s, (o, z) in enumerate(zip(o_parts, lse_parts)):
        c.tensor(f"o_parts[{s}]", o, torch.float32, (rows, Hq, d))
        c.tensor(f"lse_parts[{s}]", z, torch.float32, (Hq, rows))
    c.tensor("o_out", o_out, torch.bfloat16, (rows, Hq, d))
    c.tensor("lse_out", lse_out, torch.float32, (Hq, rows))
    c.done()
    op = (ctypes.c_void_p * n)(*[t.data_ptr() for t in o_parts])
    zp = (ctypes.c_void_p * n)(*[t.data_ptr() for t in lse_parts])
    st = lib().csbp_lse_merge(n, op, zp, rows, Hq, d, _ptr(o_out), _ptr(lse_out),
                              _stream_ptr(stream))
    _check("csbp_lse_merge", st)


def wait_selftest(budget_ns, workspace, stream=None):
    """Launch the hang-guard self-test (a bounded wait that must give up)."""
    _check("csbp_wait_selftest",
           lib().csbp_wait_selftest(int(budget_ns), _ptr(workspace), _stream_ptr(stream)))


def check_status(workspace, stream=None):
    st = lib().csbp_check_status(_ptr(workspace), _stream_ptr(stream))
    _check("csbp_check_status", st)


class BlockDiffusionAttention:
    """Owns the device work list and workspaces of one problem shape.

    forward(t) / backward(t, o) take dicts of bf16 [batch, L, H, d] CUDA
    tensors (keys as in `inputs.make_inputs`) and return fresh outputs.
    """

    def __init__(self, batch, L, M, Hq, Hkv, d, P=1, has_clean_queries=True, scale=None,
                 device="cuda", window=0, clean_causal=False, bwd_chunk=0, rank=None):
        import torch
        self.problem = make_problem(batch, L, M, Hq, Hkv, d, P, has_clean_queries, scale,
                                    window=window, clean_causal=clean_causal,
                                    bwd_chunk=bwd_chunk, rank=rank)
        bo, co, words, info = block_schedule(self.problem)
        self.block_owner, self.chunk_owner, self.info = bo, co, info
        self.work_host = words
        self.work_dev = torch.from_numpy(words).to(device)
        self.ws_fwd = _zeros(workspace_bytes(self.problem, 0), device)
        self.ws_bwd = _zeros(workspace_bytes(self.problem, 1), device)
        self.device = device
        self.shape = (batch, L, Hq, d)
        self.kv_shape = (batch, L, Hkv, d)
        self.has_clean = has_clean_queries

    def alloc_outputs(self):
        import torch
        b, L, Hq, d = self.shape
        o_clean = torch.empty(self.shape, dtype=torch.bfloat16, device=self.device) if self.has_clean else None
        o_corr = torch.empty(self.shape, dtype=torch.bfloat16, device=self.device)
        lse = torch.full((b, 2, Hq, L), float("nan"), dtype=torch.float32, device=self.device)
        return o_clean, o_corr, lse

    def alloc_grads(self):
        import torch
        g = {k: torch.empty(self.kv_shape, dtype=torch.bfloat16, device=self.device)
             for k in ("dk_clean", "dv_clean", "dk_corr", "dv_corr")}
        g["dq_corr"] = torch.empty(self.shape, dtype=torch.bfloat16, device=self.device)
        g["dq_clean"] = (torch.empty(self.shape, dtype=torch.bfloat16, device=self.device)
                         if self.has_clean else None)
        return g

    def forward(self, t, out=None, stream=None):
        o_clean, o_corr, lse = out if out is not None else _fresh(stream, self.alloc_outputs)
        attn_fwd(self.problem, t, self.work_dev, self.info, o_clean, o_corr, lse, self.ws_fwd,
                 stream)
        return o_clean, o_corr, lse

    def backward(self, t, fwd_out, grads=None, stream=None):
        o_clean, o_corr, lse = fwd_out
        g = grads if grads is not None else _fresh(stream, self.alloc_grads)
        attn_bwd(self.problem, t, self.work_dev, self.info, o_clean, o_corr, lse,
                 t.get("do_clean"), t["do_corr"], g, self.ws_bwd, stream)
        return g

    def check(self, stream=None):
        check_status(self.ws_fwd, stream)
        check_status(self.ws_bwd, stream)


# ------------------------------------------------------------ vocabulary loss
def make_ce_problem(rows, d_model, vocab, chunk_rows=0, head_grad=True, grad_scale=1.0):
    return CeProblem(int(rows), int(d_model), int(vocab), int(chunk_rows),
                     1 if head_grad else 0, float(grad_scale))


def ce_workspace_bytes(problem: CeProblem) -> int:
    return int(lib().csbp_ce_workspace_bytes(ctypes.byref(problem)))


def vocab_ce(problem, h, w, target, loss, lse, dh, dw, workspace, stream=None):
    import torch
    c = _Checks("csbp_vocab_ce")
    N, Dm, V = problem.rows, problem.d_model, problem.vocab
    c.tensor("h", h, torch.bfloat16, (N, Dm))
    c.tensor("w", w, torch.bfloat16, (V, Dm))
    c.tensor("target", target, torch.int32, (N,))
    c.tensor("loss", loss, torch.float32, (N,))
    c.tensor("lse", lse, torch.float32, (N,))
    c.tensor("dh", dh, torch.bfloat16, (N, Dm))
    if problem.head_grad:
        c.tensor("dw", dw, torch.float32, (V, Dm))
    elif dw is not None:
        raise ValueError("csbp_vocab_ce: dw must be None for a frozen head")
    c.tensor("workspace", workspace, torch.uint8, None)
    c.done()
    st = lib().csbp_vocab_ce(ctypes.byref(problem), _ptr(h), _ptr(w), _ptr(target), _ptr(loss),
                             _ptr(lse), _ptr(dh), _ptr(dw), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _check("csbp_vocab_ce", st)


class VocabCrossEntropy:
    """Owns the workspace of one LM-head cross-entropy shape.

    __call__(h, w, target) takes bf16 h [N, Dm], bf16 w [V, Dm] and int32
    target [N] on the GPU and returns (loss [N], lse [N], dh [N, Dm] bf16,
    dw [V, Dm] fp32 or None for a frozen head).
    """

    def __init__(self, rows, d_model, vocab, chunk_rows=0, head_grad=True, grad_scale=1.0,
                 device="cuda"):
        self.problem = make_ce_problem(rows, d_model, vocab, chunk_rows, head_grad, grad_scale)
        n = ce_workspace_bytes(self.problem)
        if n == 0:
            raise CsbpError("csbp_ce_workspace_bytes", -1)
        self.ws = _zeros(n, device)
        self.device = device

    def alloc_outputs(self):
        import torch
        p = self.problem
        loss = torch.empty(p.rows, dtype=torch.float32, device=self.device)
        lse = torch.empty(p.rows, dtype=torch.float32, device=self.device)
        dh = torch.empty((p.rows, p.d_model), dtype=torch.bfloat16, device=self.device)
        dw = (torch.empty((p.vocab, p.d_model), dtype=torch.float32, device=self.device)
              if p.head_grad else None)
        return loss, lse, dh, dw

    def __call__(self, h, w, target, out=None, stream=None):
        loss, lse, dh, dw = out if out is not None else _fresh(stream, self.alloc_outputs)
        vocab_ce(self.problem, h, w, target, loss, lse, dh, dw, self.ws, stream)
        return loss, lse, dh, dw

    def check(self, stream=None):
        check_status(self.ws, stream)


# ----------------------------------------------------------------- generation
# Each call takes `stream` (default: the current one).  The caller orders a stream
# that is named after what its inputs come from, and its results before their use.


class _Call:
    """Argument checks of the generation operators: dtype, shape and layout of
    every tensor first, then (in `device`) that all of them are on one CUDA
    device."""

    def __init__(self, fn):
        self.fn = fn
        self.seen = []

    def tensor(self, name, t, dtype, shape):
        """A contiguous tensor."""
        self.shaped(name, t, dtype, shape)
        if not t.is_contiguous():
            raise ValueError(f"{self.fn}: {name} must be contiguous")
        return t.data_ptr()

    def shaped(self, name, t, dtype, shape):
        if t is None:
            raise ValueError(f"{self.fn}: {name} is required")
        if t.dtype != dtype:
            raise ValueError(f"{self.fn}: {name} must be {dtype}, got {t.dtype}")
        if tuple(t.shape) != shape:
            raise ValueError(f"{self.fn}: {name} must have shape {shape}, got {tuple(t.shape)}")
        self.seen.append((name, t))

    def strided(self, name, t, shape):
        """A bf16 [batch][rows][heads][d] tensor (or [rows][heads][d]) whose
        tokens and batch entries may be strided: (pointer, token stride, batch
        stride), 0 where the dimension has one entry."""
        import torch
        self.shaped(name, t, torch.bfloat16, shape)
        st = t.stride()
        H, d = shape[-2:]
        row = H * d
        if t.numel() == 0:
            return t.data_ptr(), 0, 0
        if st[-1] != 1 or (H > 1 and st[-2] != d):
            raise ValueError(f"{self.fn}: {name} must have contiguous heads and features "
                             f"(strides [..., d, 1]), got {tuple(st)}")
        tok = st[-3] if shape[-3] > 1 else 0
        if shape[-3] > 1 and (tok < row or tok % 8):
            raise ValueError(f"{self.fn}: {name} token stride {tok} must be >= H*d = {row} and "
                             f"a multiple of 8")
        bat = st[0] if len(shape) == 4 and shape[0] > 1 else 0
        if len(shape) == 4 and shape[0] > 1 and (bat < shape[1] * (tok or row) or bat % 8):
            raise ValueError(f"{self.fn}: {name} batch entries must not interleave (batch stride "
                             f">= rows x token stride, a multiple of 8), got {bat}")
        return t.data_ptr(), tok, bat

    def device(self):
        """The index of the CUDA device that all tensors are on."""
        dev = None
        for name, t in self.seen:
            if not t.is_cuda:
                raise ValueError(f"{self.fn}: {name} must be a CUDA tensor")
            if dev is None:
                dev = t.device
            elif t.device != dev:
                raise ValueError(f"{self.fn}: {name} is on {t.device}, other tensors on {dev}")
        return dev.index


# Layouts that passed the checks, by function, problem and the (shape, strides,
# dtype, device) of every tensor: a decoding loop calls with the same few, and
# the checks in Python cost more than the launch.  Addresses are not part of it.
_LAYOUTS = {}


def _layout(fn, problem, tensors, check):
    """What `check()` returned for this layout, now or before."""
    key = (fn, problem, *[None if t is None else (t.shape, t.stride(), t.dtype, t.device)
                          for t in tensors])
    made = _LAYOUTS.get(key)
    if made is None:
        made = check()
        if len(_LAYOUTS) >= 1024:
            _LAYOUTS.clear()
        _LAYOUTS[key] = made
    return made


def _run(fn, dev, stream, tensors, *args):
    """Call the library on `stream` (default: device `dev`'s current one) with
    that device current.  The memory of `tensors` stays theirs until a stream
    that was named has done with them."""
    import torch
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"{fn}: the stream is on {stream.device}, the tensors on cuda:{dev}")
    else:
        raw = stream.cuda_stream
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    f = getattr(_lib, fn)
    if torch._C._cuda_getDevice() == dev:
        st = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = f(*args, raw)
    if st != OK:
        raise CsbpError(fn, st)


class Rotary:
    """Rotary positions of a model: `frequencies` are dim / 2 numbers in radians
    per position (theta ** (-2 i / dim) as a rule, scaled as the model has it),
    for the pairs (x_i, x_{i + dim/2}) of a head's first dim features, or
    (x_2i, x_2i+1) if `interleaved`.  dim is a multiple of 16.  Keeps them on the
    device in a form that is exact at any position."""

    def __init__(self, frequencies, interleaved=False, device="cuda"):
        import torch
        n = len(frequencies)
        if n < 8 or n % 8:
            raise ValueError(f"Rotary: the number of frequencies, dim / 2, must be a multiple of "
                             f"8, got {n}")
        turns = (ctypes.c_uint64 * n)()
        st = lib().csbp_rotary_turns((ctypes.c_double * n)(*[float(f) for f in frequencies]), n,
                                     turns)
        _check("csbp_rotary_turns", st)
        host = torch.frombuffer(turns, dtype=torch.int64).clone()
        self.turns = host.to(device)  # (pageable: the host waits for the copy)
        self.dim = 2 * n
        self.struct = RotaryStruct(self.dim, 1 if interleaved else 0, self.turns.data_ptr())
        self._ref = ctypes.byref(self.struct)


class QuantCache:
    """One layer's paged K/V cache in E4M3 with a power-of-two scale per 32
    features of a head (csbp_cache_write / csbp_cache_append / csbp_cache_read;
    PagedAttention reads it where it lies).

    Owns (or, with `storage`, wraps) the uint8 tensors k, v [pages][page_size]
    [Hkv][d] and k_scale, v_scale [pages][page_size][Hkv][d / 32].  Which pages
    a sequence has is the caller's: `table` int32 [batch][n] names them in
    order, `start` int32 [batch] is the position of row 0 of each sequence.
    """

    def __init__(self, pages, page_size, Hkv, d, device="cuda", storage=None):
        import torch
        if min(pages, page_size, Hkv) < 1 or d < 32 or d > 1024 or d % 32:
            raise ValueError("QuantCache: pages, page_size and Hkv must be positive and d a "
                             "multiple of 32 up to 1024")
        code = (pages, page_size, Hkv, d)
        scale = (pages, page_size, Hkv, d // 32)
        if storage is None:
            storage = [_zeros(s, device) for s in (code, code, scale, scale)]
        self.k, self.v, self.k_scale, self.v_scale = storage
        c = _Call("QuantCache")
        self._tensors = list(zip(("k", "v", "k_scale", "v_scale"), storage))
        ptrs = [c.tensor(n, t, torch.uint8, s)
                for (n, t), s in zip(self._tensors, (code, code, scale, scale))]
        if any(t.device != self.k.device for t in storage):
            raise ValueError("QuantCache: the storage tensors must be on one device")
        self.Hkv, self.d = Hkv, d
        self.struct = KvCache(pages, page_size, Hkv, d, *ptrs)
        self._ref = ctypes.byref(self.struct)
        self._key = (Hkv, d, str(self.k.device))

    def _check(self, fn, k, v, table, start, count, more=None):
        """(CacheRows without pointers or None, device index); `more(call)` checks
        what else the call takes."""
        import torch
        c = _Call(fn)
        if k is None or k.dim() != 4:
            raise ValueError(f"{fn}: k must be a [batch][rows][Hkv][d] tensor")
        batch, rows = k.shape[:2]
        shape = (batch, rows, self.Hkv, self.d)
        _, kt, kb = c.strided("k", k, shape)
        _, vt, vb = c.strided("v", v, shape)
        if table is None or table.dim() != 2:
            raise ValueError(f"{fn}: table must be a [batch][pages] tensor")
        c.tensor("table", table, torch.int32, (batch, table.shape[1]))
        c.tensor("start", start, torch.int32, (batch,))
        if count is not None:
            c.tensor("count", count, torch.int32, (batch,))
        c.seen += self._tensors
        if more is not None:
            more(c)
        if batch * rows == 0:
            return None, 0
        r = CacheRows(batch, rows, table.shape[1], None, None, None, (kt, vt), (kb, vb))
        return r, c.device()

    def _call(self, fn, k, v, table, start, count, stream):
        lib()
        r, dev = _layout(fn, self._key, (k, v, table, start, count),
                         lambda: self._check(fn, k, v, table, start, count))
        if r is None:
            return
        r = CacheRows.from_buffer_copy(r)
        r.table = table.data_ptr()
        r.start = start.data_ptr()
        if count is not None:
            r.count = count.data_ptr()
        _run(fn, dev, stream, (k, v, table, start, count, self.k, self.v, self.k_scale,
                               self.v_scale),
             self._ref, ctypes.byref(r), k.data_ptr(), v.data_ptr())

    def write(self, k, v, table, start, count=None, stream=None):
        """Quantise bf16 k, v [batch][rows][Hkv][d] (token and batch strides
        free) into the pages; rows i >= count[b] are not written."""
        self._call("csbp_cache_write", k, v, table, start, count, stream)

    def read(self, table, start, count=None, rows=None, out=None, stream=None):
        """bf16 (k, v) [batch][rows][Hkv][d] of positions start[b] .. ; `out`
        receives them (rows i >= count[b] keep what they hold), else two
        tensors of `rows` rows are allocated (zero beyond count)."""
        import torch
        if out is None:
            if rows is None or table is None:
                raise ValueError("csbp_cache_read: needs `rows` or `out`")
            shape = (table.shape[0], rows, self.Hkv, self.d)
            out = _fresh(stream, lambda: tuple(
                torch.zeros(shape, dtype=torch.bfloat16, device=self.k.device)
                for _ in range(2)))
        self._call("csbp_cache_read", out[0], out[1], table, start, count, stream)
        return out

    def append(self, k, v, table, start, count=None, *, rotary, q=None, out=None, stream=None):
        """`write` of k, rotated by its positions start[b] + i, and of v; q
        [batch][rows][Hq][d], if given, is rotated along.  Returns the rotated
        q: `out` (which may be q; rows i >= count[b] keep what they hold), or a
        tensor made here (zero there), or None without q."""
        import torch
        fn = "csbp_cache_append"
        lib()
        qs = AppendQueries()

        def more(c):
            nonlocal qs
            if not isinstance(rotary, Rotary):
                raise ValueError(f"{fn}: rotary must be a Rotary")
            if rotary.dim > self.d:
                raise ValueError(f"{fn}: rotary has {rotary.dim} features, a head {self.d}")
            c.seen.append(("rotary", rotary.turns))
            if q is None:
                if out is not None:
                    raise ValueError(f"{fn}: out without q")
                return
            if q.dim() != 4:
                raise ValueError(f"{fn}: q must be a [batch][rows][Hq][d] tensor")
            shape = (*k.shape[:2], q.shape[2], self.d)
            _, qt, qb = c.strided("q", q, shape)
            ot = ob = 0
            if out is not None:
                _, ot, ob = c.strided("out", out, shape)
            qs = AppendQueries(q.shape[2], 1 if out is None else 0, None, None, (qt, ot), (qb, ob))

        def check():
            return (*self._check(fn, k, v, table, start, count, more), qs)

        turns = rotary.turns if isinstance(rotary, Rotary) else None
        r, dev, qs = _layout(fn, self._key, (k, v, table, start, count, q, out, turns), check)
        if q is not None and out is None:
            out, = _fresh(stream, lambda: (
                torch.empty(q.shape, dtype=q.dtype, device=q.device),))
        if r is None:
            return out
        r = CacheRows.from_buffer_copy(r)
        r.table = table.data_ptr()
        r.start = start.data_ptr()
        if count is not None:
            r.count = count.data_ptr()
        if q is not None:
            qs = AppendQueries.from_buffer_copy(qs)
            qs.q = q.data_ptr()
            qs.out = out.data_ptr()
        _run(fn, dev, stream, (k, v, table, start, count, q, out, turns, self.k, self.v,
                               self.k_scale, self.v_scale),
             self._ref, ctypes.byref(r), rotary._ref, k.data_ptr(), v.data_ptr(),
             ctypes.byref(qs))
        return out


class PagedAttention:
    """Attention of `queries` new tokens of each of `batch` sequences over the
    pages of a QuantCache (csbp_attn_paged).  Owns the workspace of one shape,
    for all caches (layers) of that shape.

    forward(q, cache, table, length) takes bf16 q [batch][queries][Hq][d], the
    cache with the new tokens' own keys in it, int32 table [batch][table_pages]
    and int32 length [batch] (keys, the new ones included), and returns (o, lse):
    bf16 [batch][queries][Hq][d] and fp32 [batch][Hq][queries].  causal: the
    queries are the last tokens of `length` and read keys up to themselves;
    otherwise (a block being denoised) they read all of them.  window: only the
    last `window` keys up to a query's position count, and the first `sinks`.
    Calls that can overlap (two streams, two captured graphs) need handles of
    their own: they share this one's workspace.
    """

    def __init__(self, batch, queries, table_pages, page_size, Hq, Hkv, d, causal=False, window=0,
                 sinks=0, scale=None, device="cuda"):
        import torch
        self.problem = PagedProblem(batch, queries, table_pages, Hq, 1 if causal else 0, window,
                                    sinks, float(scale if scale is not None else d ** -0.5))
        self._cache = KvCache(1, page_size, Hkv, d)
        if torch.device(device).type == "cuda":
            with torch.cuda.device(device):
                n = paged_workspace_bytes(self.problem, self._cache)
        else:
            n = paged_workspace_bytes(self.problem, self._cache)
        if n == 0:
            raise CsbpError("csbp_paged_workspace_bytes", -1)
        self.ws = _zeros(n, device)
        self.device = self.ws.device
        self._key = (bytes(self.problem), page_size, Hkv, d, str(self.device))

    def alloc_outputs(self):
        import torch
        p = self.problem
        return (torch.empty((p.batch, p.queries, p.Hq, self._cache.d), dtype=torch.bfloat16,
                            device=self.device),
                torch.empty((p.batch, p.Hq, p.queries), dtype=torch.float32, device=self.device))

    def forward(self, q, cache, table, length, out=None, stream=None):
        fn = "csbp_attn_paged"
        p, mine = self.problem, self._cache
        if not isinstance(cache, QuantCache):
            raise ValueError(f"{fn}: cache must be a QuantCache")
        lib()
        o, lse = out if out is not None else (None, None)

        def check():
            import torch
            c = _Call(fn)
            got = cache.struct.page_size, cache.Hkv, cache.d
            want = mine.page_size, mine.Hkv, mine.d
            if got != want:
                raise ValueError(f"{fn}: the cache has (page_size, Hkv, d) = {got}, this handle "
                                 f"{want}")
            _, tok, bat = c.strided("q", q, (p.batch, p.queries, p.Hq, mine.d))
            c.tensor("table", table, torch.int32, (p.batch, p.table_pages))
            c.tensor("length", length, torch.int32, (p.batch,))
            if out is not None:
                c.tensor("o", o, torch.bfloat16, (p.batch, p.queries, p.Hq, mine.d))
                c.tensor("lse", lse, torch.float32, (p.batch, p.Hq, p.queries))
            c.seen += [("workspace", self.ws), *cache._tensors]
            return PagedInputs(None, tok, bat), c.device()

        inp, dev = _layout(fn, (self._key, cache._key, cache.struct.page_size),
                           (q, table, length, o, lse), check)
        if out is None:
            o, lse = _fresh(stream, self.alloc_outputs)
        inp = PagedInputs.from_buffer_copy(inp)
        inp.q = q.data_ptr()
        inp.table = table.data_ptr()
        inp.length = length.data_ptr()
        _run(fn, dev, stream, (q, table, length, o, lse, self.ws, cache.k, cache.v, cache.k_scale,
                               cache.v_scale),
             ctypes.byref(p), cache._ref, ctypes.byref(inp), o.data_ptr(), lse.data_ptr(),
             self.ws.data_ptr(), self.ws.numel())
        return o, lse

    def check(self, stream=None):
        check_status(self.ws, stream)


def paged_workspace_bytes(problem: PagedProblem, cache: KvCache) -> int:
    return int(lib().csbp_paged_workspace_bytes(ctypes.byref(problem), ctypes.byref(cache)))


class PrefixAttention:
    """Attention of `batch` sequences of `queries` tokens that share a prefix
    of prefix_len keys and have up to own_max keys of their own
    (csbp_attn_prefix).  Owns the workspace of one shape.

    forward(q, k_prefix, v_prefix, k_own, v_own, own_len) takes bf16 q
    [batch][queries][Hq][d], prefix K/V [prefix_len][Hkv][d], own K/V
    [batch][own_max][Hkv][d] and int32 own_len [batch], and returns (o, lse):
    bf16 [batch][queries][Hq][d] and fp32 [batch][Hq][queries].  causal: the
    queries are the last tokens of own_len and read own keys up to themselves;
    otherwise (a block being denoised) they read all own_len keys.  The prefix
    (own) tensors may be None when prefix_len (own_max) is 0.  The work is cut up
    for lengths of five eighths of own_max: views k[:, :m] of a larger room, with
    an own_max = m near the lengths in use, are faster than the whole room.
    Calls that can overlap (two streams, two captured graphs) need handles of
    their own: they share this one's workspace.
    """

    def __init__(self, batch, queries, prefix_len, own_max, Hq, Hkv, d, causal=False,
                 scale=None, device="cuda"):
        import torch
        self.problem = PrefixProblem(batch, queries, prefix_len, own_max, Hq, Hkv, d,
                                     1 if causal else 0,
                                     float(scale if scale is not None else d ** -0.5))
        if torch.device(device).type == "cuda":
            with torch.cuda.device(device):
                n = prefix_workspace_bytes(self.problem)
        else:
            n = prefix_workspace_bytes(self.problem)
        if n == 0:
            raise CsbpError("csbp_prefix_workspace_bytes", -1)
        self.ws = _zeros(n, device)
        self.device = self.ws.device

    def alloc_outputs(self):
        import torch
        p = self.problem
        return (torch.empty((p.batch, p.queries, p.Hq, p.d), dtype=torch.bfloat16,
                            device=self.device),
                torch.empty((p.batch, p.Hq, p.queries), dtype=torch.float32, device=self.device))

    def forward(self, q, k_prefix, v_prefix, k_own, v_own, own_len, out=None, stream=None):
        o, lse = out if out is not None else _fresh(stream, self.alloc_outputs)
        attn_prefix(self.problem, q, k_prefix, v_prefix, k_own, v_own, own_len, o, lse, self.ws,
                    stream, made_here=out is None)
        return o, lse

    def check(self, stream=None):
        check_status(self.ws, stream)


def prefix_workspace_bytes(problem: PrefixProblem) -> int:
    return int(lib().csbp_prefix_workspace_bytes(ctypes.byref(problem)))


def attn_prefix(problem, q, k_prefix, v_prefix, k_own, v_own, own_len, o, lse, workspace,
                stream=None, made_here=False):
    """csbp_attn_prefix.  `made_here`: o, lse and workspace are this module's own
    (their layout is known; the device is the workspace's)."""
    p = problem
    if not p.prefix_len:
        k_prefix = v_prefix = None
    if not p.own_max:
        k_own = v_own = own_len = None

    def check():
        import torch
        c = _Call("csbp_attn_prefix")
        pre = (p.prefix_len, p.Hkv, p.d)
        mine = (p.batch, p.own_max, p.Hkv, p.d)
        none = (None, 0, 0)
        s = [c.strided("q", q, (p.batch, p.queries, p.Hq, p.d)),
             c.strided("k_prefix", k_prefix, pre) if p.prefix_len else none,
             c.strided("v_prefix", v_prefix, pre) if p.prefix_len else none,
             c.strided("k_own", k_own, mine) if p.own_max else none,
             c.strided("v_own", v_own, mine) if p.own_max else none]
        if p.own_max:
            c.tensor("own_len", own_len, torch.int32, (p.batch,))
        c.tensor("o", o, torch.bfloat16, (p.batch, p.queries, p.Hq, p.d))
        c.tensor("lse", lse, torch.float32, (p.batch, p.Hq, p.queries))
        if workspace is None:
            raise ValueError("csbp_attn_prefix: workspace is required")
        c.tensor("workspace", workspace, torch.uint8, (workspace.numel(),))
        return (PrefixInputs(None, None, None, None, None, None, tuple(x[1] for x in s),
                             tuple(x[2] for x in s)), c.device())

    lib()
    outputs = (workspace.device,) if made_here else ()
    inp, dev = _layout("csbp_attn_prefix", (bytes(p), outputs),
                       (q, k_prefix, v_prefix, k_own, v_own, own_len) if made_here else
                       (q, k_prefix, v_prefix, k_own, v_own, own_len, o, lse, workspace), check)
    inp = PrefixInputs.from_buffer_copy(inp)
    inp.q = q.data_ptr()
    if k_prefix is not None:
        inp.k_prefix = k_prefix.data_ptr()
        inp.v_prefix = v_prefix.data_ptr()
    if k_own is not None:
        inp.k_own = k_own.data_ptr()
        inp.v_own = v_own.data_ptr()
        inp.own_len = own_len.data_ptr()
    _run("csbp_attn_prefix", dev, stream,
         (q, k_prefix, v_prefix, k_own, v_own, own_len, o, lse, workspace),
         ctypes.byref(p), ctypes.byref(inp), o.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
         workspace.numel())


def draft_verify(p, q, token, u, r, length=None, out=None, stream=None):
    """csbp_draft_verify: fp32 p [batch][drafts + 1][vocab] and q [batch]
    [drafts][vocab] (rows and batch entries may be strided), int32 token and
    fp32 u [batch][drafts], fp32 r [batch], int32 length [batch] or None.
    Returns int32 (accepted [batch], tokens [batch][drafts + 1]: the accepted
    drafts, the next token, then -1); `out` receives them if given.  q, token
    and u may be None when p has one row per sequence (plain sampling)."""
    accepted, tokens = out if out is not None else (None, None)

    def check():
        import torch
        c = _Call("csbp_draft_verify")
        if p is None or p.dim() != 3 or p.shape[1] < 1:
            raise ValueError("csbp_draft_verify: p must be a [batch][drafts + 1][vocab] tensor")
        batch, K, V = p.shape[0], p.shape[1] - 1, p.shape[2]

        def rows(name, t, n):
            """Row and batch stride of fp32 [batch][n][vocab]."""
            c.shaped(name, t, torch.float32, (batch, n, V))
            if t.numel() == 0:
                return 0, 0
            st = t.stride()
            if V > 1 and st[2] != 1:
                raise ValueError(f"csbp_draft_verify: {name} must have contiguous rows")
            row = st[1] if n > 1 else V
            if row < V:
                raise ValueError(f"csbp_draft_verify: {name} rows must not overlap (stride {row})")
            if batch > 1 and st[0] < n * row:
                raise ValueError(f"csbp_draft_verify: {name} batch entries must not interleave "
                                 f"(stride {st[0]})")
            return row, st[0] if batch > 1 else 0

        strides = rows("p", p, K + 1)
        if K:
            strides += rows("q", q, K)
            c.tensor("token", token, torch.int32, (batch, K))
            c.tensor("u", u, torch.float32, (batch, K))
        else:
            strides += (0, 0)
        c.tensor("r", r, torch.float32, (batch,))
        if length is not None:
            c.tensor("length", length, torch.int32, (batch,))
        if out is not None:
            c.tensor("accepted", accepted, torch.int32, (batch,))
            c.tensor("tokens", tokens, torch.int32, (batch, K + 1))
        dev = c.device() if batch else 0
        return VerifyProblem(batch, K, V, *strides), dev, K, (batch,), (batch, K + 1)

    lib()
    prob, dev, K, *shapes = _layout("csbp_draft_verify", out is None,
                                    (p, q, token, u, r, length, accepted, tokens), check)
    if out is None:
        import torch
        accepted, tokens = _fresh(stream, lambda: tuple(
            torch.empty(s, dtype=torch.int32, device=p.device) for s in shapes))
    if prob.batch:
        _run("csbp_draft_verify", dev, stream,
             (p, r, length, accepted, tokens) + ((q, token, u) if K else ()),
             ctypes.byref(prob), p.data_ptr(),
             q.data_ptr() if K else None, token.data_ptr() if K else None,
             u.data_ptr() if K else None, r.data_ptr(),
             None if length is None else length.data_ptr(), accepted.data_ptr(),
             tokens.data_ptr())
    return accepted, tokens
