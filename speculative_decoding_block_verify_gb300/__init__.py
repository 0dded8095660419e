"""GB300-native speculative-decoding verify sampler: Python binding of libspecverify.so.

The binding only marshals arguments: it checks tensor devices, dtypes and shapes, passes raw
device pointers and the current CUDA stream to the C ABI (``include/specverify.h``) and
raises on a nonzero return code.  Every step of the method runs in the library's CUDA
kernels; there is no fallback.  PyTorch supplies device memory and streams.

Entry points (same names as the C ABI):

* ``dspark_markov_bias``     - Markov head's low-rank previous-token logit bias
* ``dspark_markov_walk``     - the bias with the draft tokens sampled slot by slot
* ``spec_verify_tokenwise``  - token-by-token speculative sampling
* ``spec_verify_block``      - block verification
* ``spec_verify_*_reduced``  - the same over a reduced draft vocabulary (top-k draft columns)
* ``adaptive_pick_k``        - confidence head + pick how many drafts to verify
* ``spec_accept_counters``   - per-position acceptance counts (a_p, tokens per step)
* ``SpecPipeline``           - pick k -> ragged verify -> counters as one CUDA graph
* ``CostCurve``              - the online verify-cost table adaptive_pick_k reads
* ``spec_paged_attention``   - a verify block's attention over a paged key-value cache
* ``spec_cache_append``      - the block's keys and values into their pages (``reserved``: of the streams that
                               spec_cache_resize had room for)
* ``spec_cache_resize``      - pages reserved before a block and given back after its verify
* ``spec_cache_fork``        - a stream's pages shared with other streams
* ``spec_prompt_attention``  - causal attention over whole prompts, packed one behind the other
* ``spec_prompt_mark_timeout`` - what a wait that gave up has left there is cleared
* ``spec_rotate``            - rotary positions of packed rows (``RotaryTable``: their frequencies)
* ``spec_cache_append_rotated`` - a block's or a whole prompt's keys rotated into their pages, its queries rotated on the way
* ``spec_philox_uniforms``   - the verify calls' uniforms (for checking)

Every call takes ``stream`` (None: the current one).  What it makes for the caller when ``out`` is None belongs to that
stream, as if made under ``torch.cuda.stream(stream)``: a caller that reads it on another stream orders the two.

Build the library first: ``python -m speculative_decoding_block_verify_gb300.build`` (or
``__graft_entry__.build()``).
"""

import contextlib
import ctypes
import os
import struct

__all__ = [
    "dspark_markov_bias", "dspark_markov_walk", "spec_verify_tokenwise", "spec_verify_block",
    "spec_verify_tokenwise_reduced", "spec_verify_block_reduced",
    "adaptive_pick_k", "spec_accept_counters", "acceptance_rates", "SpecPipeline", "CostCurve",
    "spec_philox_uniforms", "spec_verify_launch_info",
    "spec_verify_workspace_bytes", "spec_verify_block_static",
    "spec_paged_attention", "spec_cache_append", "spec_cache_resize", "spec_cache_fork", "spec_prompt_attention",
    "spec_prompt_mark_timeout", "RotaryTable", "spec_rotate", "spec_cache_append_rotated", "lib", "lib_path", "SpecError",
    "DTYPE_F32", "DTYPE_BF16", "STATUS_NAMES", "DIAG_COLS",
]

DTYPE_F32 = 0
DTYPE_BF16 = 1
DIAG_COLS = 8
MAX_DRAFTS = 32
STATUS_NAMES = {0: "OK", 1: "BAD_TEMPERATURE", 2: "BAD_TOKEN", 3: "BAD_ROW",
                4: "ZERO_DRAFT_PROB", 5: "BAD_OFFSETS", 6: "TIMEOUT", 7: "NUMERIC",
                8: "NO_PAGES", 9: "BAD_LENGTH", 10: "BAD_PAGE", 11: "BAD_STREAM"}
EXPORTED = ["dspark_markov_bias", "dspark_markov_walk", "dspark_markov_walk_workspace_bytes",
            "spec_verify_tokenwise", "spec_verify_block",
            "spec_verify_tokenwise_reduced", "spec_verify_block_reduced",
            "adaptive_pick_k", "spec_philox_uniforms", "spec_verify_launch_info",
            "spec_verify_workspace_bytes", "spec_verify_block_static",
            "spec_accept_counters", "spec_pipeline_create", "spec_pipeline_launch",
            "spec_pipeline_destroy", "spec_cost_curve_create", "spec_cost_curve_begin",
            "spec_cost_curve_end", "spec_cost_curve_poll", "spec_cost_curve_observe",
            "spec_cost_curve_table", "spec_cost_curve_upload", "spec_cost_curve_destroy",
            "spec_paged_attention", "spec_paged_attention_workspace_bytes", "spec_cache_append",
            "spec_cache_append_reserved", "spec_cache_resize", "spec_cache_resize_workspace_bytes", "spec_cache_fork",
            "spec_prompt_attention", "spec_prompt_mark_timeout", "spec_rotary_frequencies", "spec_rotary_turns", "spec_rotate", "spec_cache_append_rotated",
            "spec_last_error", "spec_version"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None


class SpecError(RuntimeError):
    """A nonzero return code from the C ABI."""

    def __init__(self, code, msg):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class VerifyArgs(ctypes.Structure):
    """Mirror of spec_verify_args."""
    _fields_ = [
        ("B", ctypes.c_int32), ("V", ctypes.c_int32), ("kmax", ctypes.c_int32),
        ("cu_drafts", ctypes.c_void_p),
        ("draft_logits", ctypes.c_void_p), ("draft_dtype", ctypes.c_int32),
        ("target_logits", ctypes.c_void_p), ("target_dtype", ctypes.c_int32),
        ("draft_tokens", ctypes.c_void_p), ("temperature", ctypes.c_void_p),
        ("seed", ctypes.c_uint64), ("step", ctypes.c_uint64),
        ("accepted_len", ctypes.c_void_p), ("out_tokens", ctypes.c_void_p),
        ("n_emitted", ctypes.c_void_p), ("status", ctypes.c_void_p),
        ("diag", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class PipelineArgs(ctypes.Structure):
    """Mirror of spec_pipeline_args."""
    _fields_ = [
        ("hidden", ctypes.c_void_p), ("w", ctypes.c_void_p), ("head_dtype", ctypes.c_int32),
        ("bias", ctypes.c_float), ("H", ctypes.c_int32), ("verify_ms", ctypes.c_void_p),
        ("n_max", ctypes.c_int32), ("mode", ctypes.c_int32),
        ("rule", ctypes.c_int32), ("B", ctypes.c_int32), ("V", ctypes.c_int32), ("kmax", ctypes.c_int32),
        ("draft_logits", ctypes.c_void_p), ("draft_dtype", ctypes.c_int32),
        ("target_logits", ctypes.c_void_p), ("target_dtype", ctypes.c_int32),
        ("draft_tokens", ctypes.c_void_p), ("temperature", ctypes.c_void_p),
        ("seed", ctypes.c_uint64), ("step", ctypes.c_void_p),
        ("c_out", ctypes.c_void_p), ("a_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
        ("cu_drafts_out", ctypes.c_void_p), ("accepted_len", ctypes.c_void_p),
        ("out_tokens", ctypes.c_void_p), ("n_emitted", ctypes.c_void_p), ("status", ctypes.c_void_p),
        ("diag", ctypes.c_void_p), ("accept_counts", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


def lib_path():
    return os.path.join(_HERE, "_build", "libspecverify.so")


def lib():
    """Load libspecverify.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m speculative_decoding_block_verify_gb300.build`")
    L = ctypes.CDLL(path)
    vp, i32, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64
    L.dspark_markov_bias.argtypes = [vp, i32, i32, i32, vp, vp, vp, i32, i32, vp, vp]
    L.dspark_markov_walk.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, i32, i32, vp, u64, u64, vp, vp, vp, vp,
                                     ctypes.c_size_t, vp]
    L.dspark_markov_walk_workspace_bytes.argtypes = [i32]
    L.dspark_markov_walk_workspace_bytes.restype = ctypes.c_size_t
    L.spec_verify_tokenwise.argtypes = [ctypes.POINTER(VerifyArgs), vp]
    L.spec_verify_block.argtypes = [ctypes.POINTER(VerifyArgs), vp]
    L.spec_verify_block_static.argtypes = [ctypes.POINTER(VerifyArgs), vp]
    L.spec_verify_tokenwise_reduced.argtypes = [ctypes.POINTER(VerifyArgs), vp, i32, vp]
    L.spec_verify_block_reduced.argtypes = [ctypes.POINTER(VerifyArgs), vp, i32, vp]
    L.adaptive_pick_k.argtypes = [vp, vp, i32, ctypes.c_float, i32, i32, i32, vp, i32, i32,
                                  vp, vp, vp, vp, vp]
    L.spec_philox_uniforms.argtypes = [u64, u64, i32, i32, vp, vp]
    L.spec_verify_launch_info.argtypes = [ctypes.POINTER(VerifyArgs), ctypes.POINTER(i32),
                                          ctypes.POINTER(i32), ctypes.POINTER(i32)]
    L.spec_accept_counters.argtypes = [vp, vp, vp, i32, i32, vp, vp]
    L.spec_pipeline_create.argtypes = [ctypes.POINTER(PipelineArgs), ctypes.POINTER(vp)]
    L.spec_pipeline_launch.argtypes = [vp, vp]
    L.spec_pipeline_destroy.argtypes = [vp]
    L.spec_cost_curve_create.argtypes = [vp, i32, i32, i32, i32]
    L.spec_cost_curve_create.restype = vp
    L.spec_cost_curve_begin.argtypes = [vp, vp]
    L.spec_cost_curve_end.argtypes = [vp, i32, vp, vp]
    L.spec_cost_curve_poll.argtypes = [vp]
    L.spec_cost_curve_observe.argtypes = [vp, i32, ctypes.c_float]
    L.spec_cost_curve_table.argtypes = [vp, vp, vp]
    L.spec_cost_curve_upload.argtypes = [vp, vp, vp]
    L.spec_cost_curve_destroy.argtypes = [vp]
    L.spec_cost_curve_destroy.restype = None
    L.spec_verify_workspace_bytes.argtypes = [i32, i32]
    L.spec_verify_workspace_bytes.restype = ctypes.c_size_t
    L.spec_paged_attention.argtypes = [vp, vp]
    L.spec_paged_attention_workspace_bytes.argtypes = [vp]
    L.spec_paged_attention_workspace_bytes.restype = ctypes.c_size_t
    L.spec_cache_append.argtypes = [vp, vp]
    L.spec_cache_append_reserved.argtypes = [vp, vp, vp]
    L.spec_cache_resize.argtypes = [vp, vp]
    L.spec_cache_resize_workspace_bytes.argtypes = [i32, i32]
    L.spec_cache_resize_workspace_bytes.restype = ctypes.c_size_t
    L.spec_cache_fork.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    f64 = ctypes.c_double
    L.spec_prompt_attention.argtypes = [vp, vp]
    L.spec_prompt_mark_timeout.argtypes = [i32, vp]
    L.spec_rotary_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp, vp]
    L.spec_rotary_turns.argtypes = [vp, i32, vp]
    L.spec_rotate.argtypes = [vp, vp]
    L.spec_cache_append_rotated.argtypes = [vp, vp]
    L.spec_last_error.restype = ctypes.c_char_p
    L.spec_version.restype = ctypes.c_int32
    for name in ("dspark_markov_bias", "dspark_markov_walk", "spec_verify_tokenwise", "spec_verify_block", "spec_verify_block_static",
                 "spec_verify_tokenwise_reduced", "spec_verify_block_reduced",
                 "adaptive_pick_k", "spec_philox_uniforms", "spec_verify_launch_info",
                 "spec_accept_counters", "spec_pipeline_create", "spec_pipeline_launch",
                 "spec_pipeline_destroy", "spec_cost_curve_begin", "spec_cost_curve_end",
                 "spec_cost_curve_poll", "spec_cost_curve_observe", "spec_cost_curve_table",
                 "spec_cost_curve_upload", "spec_paged_attention", "spec_cache_append", "spec_cache_append_reserved",
                 "spec_cache_resize", "spec_cache_fork", "spec_prompt_attention", "spec_prompt_mark_timeout", "spec_rotary_frequencies",
                 "spec_rotary_turns", "spec_rotate", "spec_cache_append_rotated"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def _check(rc):
    if rc != 0:
        raise SpecError(rc, lib().spec_last_error().decode())


def _torch():
    import torch
    return torch


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _dev(t, name, dtype=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _made_on(stream):
    """Buffers that a call makes are its stream's: filled there, in order with the kernels, and free again for its work
    alone (the caller cannot order a fill inside the call on another stream)."""
    return contextlib.nullcontext() if stream is None else _torch().cuda.stream(stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None and t.numel() > 0 else ctypes.c_void_p(0)


def dspark_markov_bias(draft_logits, prev_tokens, W1, W2, out=None, stream=None):
    """out[r, v] = draft[r, v] + sum_j W1[prev[r], j] W2[j, v] (float32 output).

    draft_logits [rows, V] float32/bf16, prev_tokens [rows] int32, W1 [V, R], W2 [R, V]
    (same dtype).  ``out`` may be ``draft_logits`` itself when that is float32.
    """
    torch = _torch()
    _dev(draft_logits, "draft_logits")
    _dev(prev_tokens, "prev_tokens", torch.int32)
    _dev(W1, "W1")
    _dev(W2, "W2")
    rows, V = draft_logits.shape
    R = W2.shape[0]
    if W1.dtype != W2.dtype or tuple(W1.shape) != (V, R) or tuple(W2.shape) != (R, V):
        raise ValueError("W1 must be [V, R] and W2 [R, V] with one dtype")
    if prev_tokens.shape != (rows,):
        raise ValueError("prev_tokens must be [rows]")
    if out is None:
        with _made_on(stream):
            out = torch.empty((rows, V), dtype=torch.float32, device=draft_logits.device)
    _dev(out, "out", torch.float32)
    _check(lib().dspark_markov_bias(_ptr(draft_logits), _dtype_code(draft_logits), rows, V,
                                    _ptr(prev_tokens), _ptr(W1), _ptr(W2), _dtype_code(W1), R,
                                    _ptr(out), _stream(stream)))
    return out


def dspark_markov_walk(draft_logits, anchor, W1, W2, temperature, seed, step, out=None, stream=None):
    """The Markov walk: draft_logits [B, N, V] (float32/bf16), anchor [B] int32, W1 [V, R], W2
    [R, V] (one dtype), temperature [B] float32.  Returns (and reuses) ``out`` with tokens
    [B, N] int32, logits [B, N, V] float32 (the biased rows), status [B] int32, workspace."""
    torch = _torch()
    _dev(draft_logits, "draft_logits")
    _dev(anchor, "anchor", torch.int32)
    _dev(W1, "W1")
    _dev(W2, "W2")
    _dev(temperature, "temperature", torch.float32)
    B, N, V = draft_logits.shape
    R = W2.shape[0]
    if W1.dtype != W2.dtype or tuple(W1.shape) != (V, R) or tuple(W2.shape) != (R, V):
        raise ValueError("W1 must be [V, R] and W2 [R, V] with one dtype")
    if anchor.shape != (B,) or temperature.shape != (B,):
        raise ValueError("anchor and temperature must be [B]")
    dev = draft_logits.device
    if out is None:
        with _made_on(stream):
            out = {"tokens": torch.empty((B, N), dtype=torch.int32, device=dev),
                   "logits": torch.empty((B, N, V), dtype=torch.float32, device=dev),
                   "status": torch.empty(B, dtype=torch.int32, device=dev),
                   "workspace": torch.empty(max(int(lib().dspark_markov_walk_workspace_bytes(B)), 16),
                                            dtype=torch.uint8, device=dev)}
    _check(lib().dspark_markov_walk(_ptr(draft_logits), _dtype_code(draft_logits), B, N, V, _ptr(anchor),
                                    _ptr(W1), _ptr(W2), _dtype_code(W1), R, _ptr(temperature),
                                    int(seed) & 0xFFFFFFFFFFFFFFFF, int(step) & 0xFFFFFFFFFFFFFFFF,
                                    _ptr(out["tokens"]), _ptr(out["logits"]), _ptr(out["status"]),
                                    _ptr(out["workspace"]), out["workspace"].numel(), _stream(stream)))
    return out


def _verify(fn, cu_drafts, draft_logits, target_logits, draft_tokens, temperature, kmax, seed,
            step, out=None, diag=False, stream=None, workspace=True, t2d=None):
    """Marshals one verify call.  ``out`` (returned, and reusable by later calls of the same B
    and kmax on the same stream) holds the four result tensors and the device workspace; a
    workspace the caller puts in ``out["workspace"]`` must have been zero-filled before its
    first use (the one allocated here is), since the kernels keep per-row counters there that
    every call leaves at zero."""
    torch = _torch()
    _dev(cu_drafts, "cu_drafts", torch.int32)
    _dev(target_logits, "target_logits")
    _dev(draft_logits, "draft_logits")
    _dev(draft_tokens, "draft_tokens", torch.int32)
    _dev(temperature, "temperature", torch.float32)
    B = cu_drafts.numel() - 1
    V = target_logits.shape[1]
    if t2d is not None:
        _dev(t2d, "t2d", torch.int32)
        if t2d.numel() != V:
            raise ValueError("t2d must be [V]")
        if draft_logits.dim() != 2:
            raise ValueError("draft_logits must be [rows, K]")
    elif draft_logits.dim() != 2 or (draft_logits.shape[0] > 0 and draft_logits.shape[1] != V):
        raise ValueError("draft_logits must be [rows, V]")
    if temperature.numel() != B:
        raise ValueError("temperature must be [B]")
    dev = target_logits.device
    if out is None:
        with _made_on(stream):
            out = {
                "accepted_len": torch.empty(B, dtype=torch.int32, device=dev),
                "out_tokens": torch.empty((B, kmax + 1), dtype=torch.int32, device=dev),
                "n_emitted": torch.empty(B, dtype=torch.int32, device=dev),
                "status": torch.empty(B, dtype=torch.int32, device=dev),
            }
            if diag:
                out["diag"] = torch.empty((target_logits.shape[0], DIAG_COLS), dtype=torch.float32,
                                          device=dev)
    ws = None
    if workspace:
        need = spec_verify_workspace_bytes(B, kmax)
        ws = out.get("workspace")
        if ws is None or ws.numel() < need:
            # zero-filled once: every call leaves the row counters it used at zero
            with _made_on(stream):
                ws = out["workspace"] = torch.zeros(max(need, 16), dtype=torch.uint8, device=dev)
    a = VerifyArgs()
    a.B, a.V, a.kmax = B, V, kmax
    a.cu_drafts = cu_drafts.data_ptr()
    a.draft_logits = draft_logits.data_ptr() if draft_logits.numel() else None
    a.draft_dtype = _dtype_code(draft_logits)
    a.target_logits = target_logits.data_ptr()
    a.target_dtype = _dtype_code(target_logits)
    a.draft_tokens = draft_tokens.data_ptr() if draft_tokens.numel() else None
    a.temperature = temperature.data_ptr()
    a.seed = int(seed) & 0xFFFFFFFFFFFFFFFF
    a.step = int(step) & 0xFFFFFFFFFFFFFFFF
    a.accepted_len = out["accepted_len"].data_ptr()
    a.out_tokens = out["out_tokens"].data_ptr()
    a.n_emitted = out["n_emitted"].data_ptr()
    a.status = out["status"].data_ptr()
    a.diag = out["diag"].data_ptr() if out.get("diag") is not None else None
    a.workspace = ws.data_ptr() if ws is not None else None
    a.workspace_bytes = ws.numel() if ws is not None else 0
    if t2d is not None:
        _check(fn(ctypes.byref(a), _ptr(t2d), int(draft_logits.shape[1]), _stream(stream)))
    else:
        _check(fn(ctypes.byref(a), _stream(stream)))
    return out


def spec_verify_tokenwise(cu_drafts, draft_logits, target_logits, draft_tokens, temperature,
                          kmax, seed, step, out=None, diag=False, stream=None):
    """Token-by-token speculative sampling (see include/specverify.h)."""
    return _verify(lib().spec_verify_tokenwise, cu_drafts, draft_logits, target_logits,
                   draft_tokens, temperature, kmax, seed, step, out, diag, stream)


def spec_verify_block(cu_drafts, draft_logits, target_logits, draft_tokens, temperature, kmax,
                      seed, step, out=None, diag=False, stream=None):
    """Block verification (see include/specverify.h)."""
    return _verify(lib().spec_verify_block, cu_drafts, draft_logits, target_logits,
                   draft_tokens, temperature, kmax, seed, step, out, diag, stream)


def spec_verify_tokenwise_reduced(cu_drafts, draft_logits, t2d, target_logits, draft_tokens, temperature,
                                  kmax, seed, step, out=None, diag=False, stream=None):
    """Token-wise verify with draft rows over a reduced draft vocabulary: draft_logits [rows, K],
    t2d [V] int32 (the draft id of each target column, -1 outside the draft vocabulary)."""
    return _verify(lib().spec_verify_tokenwise_reduced, cu_drafts, draft_logits, target_logits,
                   draft_tokens, temperature, kmax, seed, step, out, diag, stream, t2d=t2d)


def spec_verify_block_reduced(cu_drafts, draft_logits, t2d, target_logits, draft_tokens, temperature, kmax,
                              seed, step, out=None, diag=False, stream=None):
    """Block verification with draft rows over a reduced draft vocabulary (see
    spec_verify_tokenwise_reduced)."""
    return _verify(lib().spec_verify_block_reduced, cu_drafts, draft_logits, target_logits,
                   draft_tokens, temperature, kmax, seed, step, out, diag, stream, t2d=t2d)


def spec_verify_block_static(cu_drafts, draft_logits, target_logits, draft_tokens, temperature,
                             kmax, seed, step, out=None, diag=False, stream=None):
    """Block verification on the library's fixed device workspace: no workspace is allocated
    or passed (see include/specverify.h for its capacity and ordering rule)."""
    return _verify(lib().spec_verify_block_static, cu_drafts, draft_logits, target_logits,
                   draft_tokens, temperature, kmax, seed, step, out, diag, stream, workspace=False)


def adaptive_pick_k(hidden, w, bias, verify_ms, mode=0, out=None, stream=None):
    """Confidence head + pick k.  hidden [B, kmax, H], w [H] (float32/bf16, same dtype),
    verify_ms [n_max + 1] float32.  Returns dict c [B, kmax], a [B, kmax], k [B], cu [B+1]."""
    torch = _torch()
    _dev(hidden, "hidden")
    _dev(w, "w")
    _dev(verify_ms, "verify_ms", torch.float32)
    if w.dtype != hidden.dtype:
        raise TypeError("hidden and w must share a dtype")
    B, kmax, H = hidden.shape
    if w.shape != (H,):
        raise ValueError("w must be [H]")
    dev = hidden.device
    if out is None:
        with _made_on(stream):
            out = {"c": torch.empty((B, kmax), dtype=torch.float32, device=dev),
                   "a": torch.empty((B, kmax), dtype=torch.float32, device=dev),
                   "k": torch.empty(B, dtype=torch.int32, device=dev),
                   "cu": torch.empty(B + 1, dtype=torch.int32, device=dev)}
    _check(lib().adaptive_pick_k(_ptr(hidden), _ptr(w), _dtype_code(hidden), float(bias), B, kmax,
                                 H, _ptr(verify_ms), verify_ms.numel() - 1, int(mode),
                                 _ptr(out["c"]), _ptr(out["a"]), _ptr(out["k"]), _ptr(out["cu"]),
                                 _stream(stream)))
    return out


def spec_accept_counters(accepted_len, status, cu_drafts, kmax, counts=None, stream=None):
    """Adds one batch's per-position acceptance counts to ``counts`` [2 kmax + 1] (uint64 as
    int64, device; allocated zeroed when None) and returns it: counts[0] = verified streams,
    counts[p] = accepted at position p, counts[kmax + p] = offered at position p."""
    torch = _torch()
    _dev(accepted_len, "accepted_len", torch.int32)
    _dev(status, "status", torch.int32)
    _dev(cu_drafts, "cu_drafts", torch.int32)
    B = status.numel()
    if counts is None:
        with _made_on(stream):
            counts = torch.zeros(2 * kmax + 1, dtype=torch.int64, device=status.device)
    _dev(counts, "counts", torch.int64)
    if counts.numel() != 2 * kmax + 1:
        raise ValueError("counts must have 2 kmax + 1 entries")
    _check(lib().spec_accept_counters(_ptr(accepted_len), _ptr(status), _ptr(cu_drafts), B, kmax,
                                      _ptr(counts), _stream(stream)))
    return counts


def acceptance_rates(counts, kmax):
    """(a_p for p = 1..kmax, marginal a_p / a_{p-1}, tokens per step = 1 + sum a_p) from the
    accumulated counts (P1 §6 "The arithmetic you need before tuning k")."""
    c = [int(v) for v in counts.cpu().tolist()]
    steps = max(c[0], 1)
    a = [c[p] / steps for p in range(1, kmax + 1)]
    marg = [a[0]] + [(a[p] / a[p - 1]) if a[p - 1] > 0 else 0.0 for p in range(1, kmax)]
    return a, marg, 1.0 + sum(a)


class SpecPipeline:
    """pick k -> verify each stream's first k_b drafts -> acceptance counters -> step + 1, as
    one CUDA graph (spec_pipeline_create / launch / destroy).  Inputs are the dense layout:
    draft_logits [B, kmax, V], target_logits [B, kmax + 1, V], draft_tokens [B, kmax]; the
    confidence head's hidden [B, kmax, H], w [H] and verify_ms [n_max + 1].  ``step`` is the
    first launch's Philox step; each launch adds 1.  The outputs (``out`` dict) and the
    counters are device tensors that every launch overwrites (counters accumulate)."""

    def __init__(self, hidden, w, bias, verify_ms, draft_logits, target_logits, draft_tokens,
                 temperature, rule=1, mode=0, seed=0, step=0, diag=False, counters=True):
        torch = _torch()
        for t, n in ((hidden, "hidden"), (w, "w"), (draft_logits, "draft_logits"),
                     (target_logits, "target_logits")):
            _dev(t, n)
        _dev(verify_ms, "verify_ms", torch.float32)
        _dev(draft_tokens, "draft_tokens", torch.int32)
        _dev(temperature, "temperature", torch.float32)
        B, kmax, V = draft_logits.shape
        if tuple(target_logits.shape) != (B, kmax + 1, V) or tuple(draft_tokens.shape) != (B, kmax):
            raise ValueError("target_logits must be [B, kmax + 1, V] and draft_tokens [B, kmax]")
        if hidden.shape[:2] != (B, kmax) or w.shape != (hidden.shape[2],) or w.dtype != hidden.dtype:
            raise ValueError("hidden must be [B, kmax, H] and w [H] of hidden's dtype")
        dev = draft_logits.device
        self.kmax = kmax
        self.out = {
            "c": torch.empty((B, kmax), dtype=torch.float32, device=dev),
            "a": torch.empty((B, kmax), dtype=torch.float32, device=dev),
            "k": torch.empty(B, dtype=torch.int32, device=dev),
            "cu": torch.empty(B + 1, dtype=torch.int32, device=dev),
            "accepted_len": torch.empty(B, dtype=torch.int32, device=dev),
            "out_tokens": torch.empty((B, kmax + 1), dtype=torch.int32, device=dev),
            "n_emitted": torch.empty(B, dtype=torch.int32, device=dev),
            "status": torch.empty(B, dtype=torch.int32, device=dev),
        }
        if diag:
            self.out["diag"] = torch.empty((B * (kmax + 1), DIAG_COLS), dtype=torch.float32, device=dev)
        self.counts = torch.zeros(2 * kmax + 1, dtype=torch.int64, device=dev) if counters else None
        self.step = torch.tensor([int(step)], dtype=torch.int64, device=dev)
        self.workspace = torch.zeros(max(spec_verify_workspace_bytes(B, kmax), 16), dtype=torch.uint8,
                                     device=dev)
        self._keep = (hidden, w, verify_ms, draft_logits, target_logits, draft_tokens, temperature)
        a = PipelineArgs()
        a.hidden, a.w, a.head_dtype = hidden.data_ptr(), w.data_ptr(), _dtype_code(hidden)
        a.bias, a.H, a.verify_ms, a.n_max, a.mode = float(bias), hidden.shape[2], verify_ms.data_ptr(), \
            verify_ms.numel() - 1, int(mode)
        a.rule, a.B, a.V, a.kmax = int(rule), B, V, kmax
        a.draft_logits, a.draft_dtype = draft_logits.data_ptr(), _dtype_code(draft_logits)
        a.target_logits, a.target_dtype = target_logits.data_ptr(), _dtype_code(target_logits)
        a.draft_tokens, a.temperature = draft_tokens.data_ptr(), temperature.data_ptr()
        a.seed, a.step = int(seed) & 0xFFFFFFFFFFFFFFFF, self.step.data_ptr()
        o = self.out
        a.c_out, a.a_out, a.k_out, a.cu_drafts_out = (o[k].data_ptr() for k in ("c", "a", "k", "cu"))
        a.accepted_len, a.out_tokens, a.n_emitted, a.status = (
            o[k].data_ptr() for k in ("accepted_len", "out_tokens", "n_emitted", "status"))
        a.diag = o["diag"].data_ptr() if diag else None
        a.accept_counts = self.counts.data_ptr() if counters else None
        a.workspace, a.workspace_bytes = self.workspace.data_ptr(), self.workspace.numel()
        self._handle = ctypes.c_void_p()
        _check(lib().spec_pipeline_create(ctypes.byref(a), ctypes.byref(self._handle)))

    def launch(self, stream=None):
        """One verify step (one graph launch on the current or given stream)."""
        _check(lib().spec_pipeline_launch(self._handle, _stream(stream)))
        return self.out

    def close(self):
        if self._handle:
            _check(lib().spec_pipeline_destroy(self._handle))
            self._handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class CostCurve:
    """The online verify-cost curve (P3 "Teaching the Speculator What a Draft Costs", "What we
    changed" and "Reproduce"): CUDA-event pairs around real verify steps, read without waiting,
    rolling medians per token count laid over the boot curve every ``rebuild_every``
    observations.  ``boot_ms`` is a host sequence of n_max + 1 floats (index = token count).

    ``begin()`` / ``end(num_tokens, device_count=None)`` bracket one verify step on the current
    (or given) stream; a ``device_count`` int32 CUDA tensor (one element) adds its value to the
    count after the step.  ``poll()`` folds in finished steps, ``table()`` returns the current
    table (a list) and ``upload(device_table)`` queues its copy into a float32 CUDA tensor."""

    def __init__(self, boot_ms, window=32, min_samples=3, rebuild_every=32):
        boot = (ctypes.c_float * len(boot_ms))(*[float(v) for v in boot_ms])
        self.n_max = len(boot_ms) - 1
        self._handle = lib().spec_cost_curve_create(boot, self.n_max, int(window), int(min_samples),
                                                     int(rebuild_every))
        if not self._handle:
            raise SpecError(-1, lib().spec_last_error().decode())

    def begin(self, stream=None):
        _check(lib().spec_cost_curve_begin(self._handle, _stream(stream)))

    def end(self, num_tokens=0, device_count=None, stream=None):
        if device_count is not None:
            _dev(device_count, "device_count", _torch().int32)
        _check(lib().spec_cost_curve_end(self._handle, int(num_tokens), _ptr(device_count), _stream(stream)))

    def poll(self):
        _check(lib().spec_cost_curve_poll(self._handle))

    def observe(self, num_tokens, ms):
        _check(lib().spec_cost_curve_observe(self._handle, int(num_tokens), float(ms)))

    def table(self):
        """(table as a list of n_max + 1 floats, {observations, rebuilds, dropped, pending})."""
        out = (ctypes.c_float * (self.n_max + 1))()
        cnt = (ctypes.c_int64 * 4)()
        _check(lib().spec_cost_curve_table(self._handle, out, cnt))
        return list(out), dict(zip(("observations", "rebuilds", "dropped", "pending"), list(cnt)))

    def upload(self, device_table, stream=None):
        _dev(device_table, "device_table", _torch().float32)
        if device_table.numel() != self.n_max + 1:
            raise ValueError("device_table must hold n_max + 1 floats")
        _check(lib().spec_cost_curve_upload(self._handle, _ptr(device_table), _stream(stream)))

    def close(self):
        if self._handle:
            lib().spec_cost_curve_destroy(self._handle)
            self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def spec_verify_workspace_bytes(B, kmax):
    """Device workspace bytes a verify call over B streams with up to kmax drafts needs."""
    return int(lib().spec_verify_workspace_bytes(int(B), int(kmax)))


def spec_verify_launch_info(B, V, kmax, draft_dtype=DTYPE_BF16, target_dtype=DTYPE_BF16,
                            aligned=True):
    """(cluster_size, resident_clusters, elems_per_load) a verify call of this shape uses."""
    a = VerifyArgs()
    a.B, a.V, a.kmax = B, V, kmax
    a.draft_dtype, a.target_dtype = draft_dtype, target_dtype
    a.draft_logits = a.target_logits = 0 if aligned else 2
    c, r, e = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(lib().spec_verify_launch_info(ctypes.byref(a), ctypes.byref(c), ctypes.byref(r),
                                         ctypes.byref(e)))
    return c.value, r.value, e.value


def spec_philox_uniforms(seed, step, n_streams, n_slots, device="cuda", stream=None):
    """[n_streams, n_slots, 2] float64: (acceptance, sampling) uniforms of every (stream, slot)."""
    torch = _torch()
    with _made_on(stream):
        out = torch.empty((n_streams, n_slots, 2), dtype=torch.float64, device=device)
    _check(lib().spec_philox_uniforms(int(seed) & 0xFFFFFFFFFFFFFFFF, int(step) & 0xFFFFFFFFFFFFFFFF,
                                      n_streams, n_slots, _ptr(out), _stream(stream)))
    return out


# ---------------------------------------------------------------------------------------------
# The paged key-value cache.  These calls sit in a decode loop's every layer, so their argument
# structs are packed in one go (native alignment, as the C compiler lays them out).
# ---------------------------------------------------------------------------------------------
_ATTENTION = struct.Struct("@11i f 4P 2q 5P N")  # spec_attention_args
_APPEND = struct.Struct("@8i 5P 3q 3P")          # spec_append_args
_RESIZE = struct.Struct("@5i q 10P N")           # spec_resize_args
_PROMPT = struct.Struct("@7i f q 4P 3q 2P")      # spec_prompt_args
_ROTATE = struct.Struct("@5i f q 3P q P q")      # spec_rotate_args
_APPEND_ROTATED = struct.Struct("@12i f 8P 4q 2P 2q 3P")   # spec_append_rotated_args


_T = None       # torch, once a cache call has run
_I32 = None
_CODES = {}     # dtype -> SPEC_DTYPE_*
_ONE_DEVICE = False   # every CUDA tensor and stream is the current device's


def _cache_torch():
    global _T, _I32, _CODES, _ONE_DEVICE
    import torch
    _ONE_DEVICE = torch.cuda.device_count() == 1
    _CODES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
    _I32 = torch.int32
    _T = torch
    return torch


def _wrong(t, name, device, dtype, shape):
    """Raises what is wrong with a tensor that should be dense, of this device, dtype and shape."""
    if not isinstance(t, _T.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on another device")


def _on(t, name, device, dtype, shape):
    """The pointer of a dense tensor of this device, dtype and shape."""
    if t.get_device() != device or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _wrong(t, name, device, dtype, shape)
    return t.data_ptr()


def _packed(t, name, device, dtype, heads, D):
    """(pointer, row stride, rows) of [rows, heads, D] with dense rows (a slice of a wider projection)."""
    shape = t.shape
    if t.get_device() == device and t.dtype is dtype and len(shape) == 3:
        rows, h, d = shape
        row, head, one = t.stride()
        dense = heads * D
        if h == heads and d == D and one == 1 and (head == D or heads == 1) and (row >= dense or rows <= 1):
            return t.data_ptr(), row if row > dense else dense, rows
    if t.get_device() != device:
        raise TypeError(f"{name} must be a CUDA tensor on the cache's device")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} like the cache, got {t.dtype}")
    if len(shape) != 3 or shape[1] != heads or shape[2] != D:
        raise ValueError(f"{name} must be [rows, {heads}, {D}], got {list(shape)}")
    raise ValueError(f"{name} must have dense rows of heads * D elements")


def _rows_into(t, name, device, dtype, rows, heads, D):
    """(pointer, row stride) of an output [rows, heads, D] with dense rows."""
    if t.is_contiguous() and t.dtype is dtype and t.get_device() == device and t.shape == (rows, heads, D):
        return t.data_ptr(), heads * D
    if len(t.shape) == 3 and t.shape[0] != rows:
        raise ValueError(f"{name} must have {rows} rows, got {t.shape[0]}")
    return _packed(t, name, device, dtype, heads, D)[:2]


def _layer_of(k_pages, v_pages):
    """(device, dtype code, pointers, shape) of one layer's pool."""
    shape, device, dtype = k_pages.shape, k_pages.get_device(), k_pages.dtype
    if device < 0 or v_pages.get_device() != device:
        raise TypeError("k_pages and v_pages must be CUDA tensors on one device")
    if len(shape) != 4 or shape != v_pages.shape or dtype is not v_pages.dtype:
        raise ValueError("k_pages and v_pages must be [num_pages, Hkv, page_size, D] of one dtype")
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("k_pages and v_pages must be contiguous")
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    return device, code, k_pages.data_ptr(), v_pages.data_ptr(), shape


def _blocks_of(device, page_table, length, cu_drafts, rows, kmax):
    """(B, max_pages, pointers of cu_drafts, length, page_table) of packed blocks."""
    shape = page_table.shape
    if len(shape) != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B = shape[0]
    if cu_drafts is None:
        cu = 0
        if rows != B * (kmax + 1):
            raise ValueError("without cu_drafts there are B * (kmax + 1) rows")
    else:
        cu = _on(cu_drafts, "cu_drafts", device, _I32, (B + 1,))
    return (B, shape[1], cu, _on(length, "length", device, _I32, (B,)), _on(page_table, "page_table", device, _I32, shape))


def _raw_stream(stream, device):
    """The stream to launch on.  Launches go to the current device, so the tensors and the stream have to be its."""
    if not _ONE_DEVICE:
        current = _T._C._cuda_getDevice()
        if device != current:
            raise ValueError(f"the tensors are on cuda:{device}, the current device is cuda:{current}")
        if stream is not None and stream.device_index != device:
            raise ValueError(f"the tensors are on cuda:{device}, the stream on cuda:{stream.device_index}")
    return _T._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _space(ws, device):
    """(pointer, bytes) of a workspace."""
    if ws.get_device() != device or not ws.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA tensor on the cache's device")
    return ws.data_ptr(), ws.nbytes


def spec_paged_attention(q, k_pages, v_pages, page_table, length, cu_drafts, kmax, scale, window=0, sinks=0,
                         out=None, stream=None):
    """Attention of every stream's block (its drafts and the token before them) over its pages.

    q [rows, Hq, D] (rows may be slices of a wider projection), k_pages and v_pages [num_pages, Hkv,
    page_size, D] of q's dtype (float32/bf16), page_table [B, max_pages], length [B] (tokens before the
    block) and cu_drafts [B + 1] int32 (None: kmax drafts each; kmax = 0 is plain decoding).  window > 0
    keeps the last ``window`` positions of each row and the first ``sinks`` of its stream.  Returns
    (and reuses) ``out`` with out [rows, Hq, D], status [B], workspace.  A call that reports TIMEOUT leaves a mark in the
    workspace: the calls after it report TIMEOUT as well until the first 256 bytes are zeroed."""
    torch = _T or _cache_torch()
    device, code, kp, vp, (num_pages, Hkv, page_size, D) = _layer_of(k_pages, v_pages)
    shape = q.shape
    if len(shape) != 3 or shape[1] % Hkv != 0:
        raise ValueError("q must be [rows, Hq, D] with Hq a multiple of Hkv")
    rows, Hq, _ = shape
    qp, stride, _ = _packed(q, "q", device, k_pages.dtype, Hq, D)
    B, max_pages, cu, lp, tp = _blocks_of(device, page_table, length, cu_drafts, rows, kmax)
    L = _lib or lib()
    if out is None:
        # the first 256 bytes of the workspace start at zero and every call leaves them so (but one that reports TIMEOUT)
        need = L.spec_paged_attention_workspace_bytes(_ATTENTION.pack(
            B, kmax, Hq, Hkv, D, page_size, num_pages, max_pages, code, window, sinks, scale, cu, lp, tp, qp, stride, rows,
            kp, vp, 0, 0, 0, 0))
        with _made_on(stream):
            out = {"out": torch.empty((rows, Hq, D), dtype=q.dtype, device=q.device),
                   "status": torch.empty(B, dtype=torch.int32, device=q.device),
                   "workspace": torch.zeros(max(int(need), 16), dtype=torch.uint8, device=q.device)}
    ws, size = _space(out["workspace"], device)
    rc = L.spec_paged_attention(_ATTENTION.pack(
        B, kmax, Hq, Hkv, D, page_size, num_pages, max_pages, code, window, sinks, scale, cu, lp, tp, qp, stride, rows, kp, vp,
        _on(out["out"], "out", device, q.dtype, shape), _on(out["status"], "status", device, _I32, (B,)),
        ws, size), _raw_stream(stream, device))
    if rc != 0:
        _check(rc)
    return out


def spec_cache_append(k, v, k_pages, v_pages, page_table, length, cu_drafts, kmax, out=None, stream=None, reserved=None):
    """Writes the block's k and v [rows, Hkv, D] (slices of a wider projection may be passed) to their
    positions in one layer's pages; the other arguments as in spec_paged_attention.  With ``reserved`` (the status of
    the spec_cache_resize that made the room) a stream that has none there is left alone and reports that status: what
    keeps one that found no free page (NO_PAGES) off a page that it still shares.  Returns (and reuses) ``out`` with
    status [B]."""
    torch = _T or _cache_torch()
    device, code, kp, vp, (num_pages, Hkv, page_size, D) = _layer_of(k_pages, v_pages)
    dtype = k_pages.dtype
    nk, ks, rows = _packed(k, "k", device, dtype, Hkv, D)
    nv, vs, v_rows = _packed(v, "v", device, dtype, Hkv, D)
    if v_rows != rows:
        raise ValueError("k and v must have the same rows")
    B, max_pages, cu, lp, tp = _blocks_of(device, page_table, length, cu_drafts, rows, kmax)
    if out is None:
        with _made_on(stream):
            out = {"status": torch.empty(B, dtype=torch.int32, device=k.device)}
    args = _APPEND.pack(B, kmax, Hkv, D, page_size, num_pages, max_pages, code, cu, lp, tp, nk, nv, ks, vs, rows, kp, vp,
                        _on(out["status"], "status", device, _I32, (B,)))
    L = _lib or lib()
    if reserved is None:
        rc = L.spec_cache_append(args, _raw_stream(stream, device))
    else:
        rc = L.spec_cache_append_reserved(args, _on(reserved, "reserved", device, _I32, (B,)), _raw_stream(stream, device))
    if rc != 0:
        _check(rc)
    return out


def _book_of(page_table, held, length, ref_count):
    """(device, B, max_pages, num_pages, pointers) of a cache's bookkeeping."""
    shape, pages = page_table.shape, ref_count.shape
    if len(shape) != 2 or len(pages) != 1:
        raise ValueError("page_table must be [B, max_pages] and ref_count [num_pages]")
    device, B = page_table.get_device(), shape[0]
    if device < 0:
        raise TypeError("page_table must be a CUDA tensor")
    return (device, B, shape[1], pages[0], _on(page_table, "page_table", device, _I32, shape),
            _on(held, "held", device, _I32, (B,)), _on(length, "length", device, _I32, (B,)),
            _on(ref_count, "ref_count", device, _I32, pages))


def spec_cache_resize(k_pool, v_pool, page_table, held, length, ref_count, advance=None, room=None, out=None,
                      stream=None):
    """length += advance (n_emitted of a verify call, or negative to roll back), then every stream
    holds the pages of length + room tokens.  k_pool and v_pool [layers, num_pages, Hkv, page_size,
    D]; page_table [B, max_pages], held, length [B] and ref_count [num_pages] int32 are updated in
    place; advance and room [B] int32 or None.  Returns (and reuses) ``out`` with status [B], workspace."""
    torch = _T or _cache_torch()
    device, B, max_pages, num_pages, tp, hp, lp, rp = _book_of(page_table, held, length, ref_count)
    shape, dtype = k_pool.shape, k_pool.dtype
    if len(shape) != 5 or shape[1] != num_pages:
        raise ValueError("k_pool and v_pool must be [layers, num_pages, Hkv, page_size, D]")
    if dtype not in _CODES:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    page_size = shape[3]
    page_bytes = shape[2] * page_size * shape[4] * (4 if dtype is torch.float32 else 2)
    kp = _on(k_pool, "k_pool", device, dtype, shape)
    vp = _on(v_pool, "v_pool", device, dtype, shape)
    ap = 0 if advance is None else _on(advance, "advance", device, _I32, (B,))
    mp = 0 if room is None else _on(room, "room", device, _I32, (B,))
    L = _lib or lib()
    if out is None:
        need = max(int(L.spec_cache_resize_workspace_bytes(B, num_pages)), 16)
        with _made_on(stream):
            out = {"status": torch.empty(B, dtype=torch.int32, device=page_table.device),
                   "workspace": torch.empty(need, dtype=torch.uint8, device=page_table.device)}
    ws, size = _space(out["workspace"], device)
    rc = L.spec_cache_resize(_RESIZE.pack(
        B, page_size, num_pages, max_pages, shape[0], page_bytes, ap, mp, tp, hp, lp, rp, kp, vp,
        _on(out["status"], "status", device, _I32, (B,)), ws, size), _raw_stream(stream, device))
    if rc != 0:
        _check(rc)
    return out


def spec_cache_fork(src, dst, page_table, held, length, ref_count, page_size, out=None, stream=None):
    """Stream dst[e] becomes a continuation of stream src[e] (src, dst [n] int32): it gives up its pages
    and shares those of src's tokens; spec_cache_resize copies a shared page before it is written
    into.  Returns (and reuses) ``out`` with status [n]."""
    torch = _T or _cache_torch()
    device, B, max_pages, num_pages, tp, hp, lp, rp = _book_of(page_table, held, length, ref_count)
    n = src.numel()
    sp = _on(src, "src", device, _I32, (n,))
    dp = _on(dst, "dst", device, _I32, (n,))
    if out is None:
        with _made_on(stream):
            out = {"status": torch.empty(n, dtype=torch.int32, device=page_table.device)}
    rc = (_lib or lib()).spec_cache_fork(sp, dp, n, B, page_size, num_pages, max_pages, tp, hp, lp, rp,
                                         _on(out["status"], "status", device, _I32, (n,)), _raw_stream(stream, device))
    if rc != 0:
        _check(rc)
    return out


# ---------------------------------------------------------------------------------------------
# Prompts and rotary positions
# ---------------------------------------------------------------------------------------------
def spec_prompt_attention(q, k, v, cu_rows, scale, window=0, sinks=0, out=None, stream=None):
    """Causal attention over whole prompts, packed one behind the other.

    q [rows, Hq, D], k and v [rows, Hkv, D] of one dtype (float32/bf16; rows may be slices of a wider projection, on 16-byte
    boundaries); prompt b has rows cu_rows[b] .. cu_rows[b + 1] - 1 (cu_rows [B + 1] int32; None: one prompt of all rows).
    window and sinks as in spec_paged_attention.  Returns (and reuses) ``out`` with out [rows, Hq, D], status [B].  A call that reports TIMEOUT leaves
    a mark on the device: the calls after it report TIMEOUT as well until spec_prompt_mark_timeout clears it."""
    torch = _T or _cache_torch()
    shape, device, dtype = q.shape, q.get_device(), q.dtype
    if device < 0:
        raise TypeError("q must be a CUDA tensor")
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    if len(shape) != 3 or k.dim() != 3:
        raise ValueError("q must be [rows, Hq, D] and k [rows, Hkv, D]")
    rows, Hq, D = shape
    Hkv = k.size(1)
    qp, qs, _ = _packed(q, "q", device, dtype, Hq, D)
    kp, ks, k_rows = _packed(k, "k", device, dtype, Hkv, D)
    vp, vs, v_rows = _packed(v, "v", device, dtype, Hkv, D)
    if k_rows != rows or v_rows != rows:
        raise ValueError("q, k and v must have the same rows")
    if cu_rows is None:
        B, cu = 1, 0
    else:
        B = cu_rows.numel() - 1
        if B < 0:
            raise ValueError("cu_rows must be [B + 1]")
        cu = _on(cu_rows, "cu_rows", device, _I32, (B + 1,))
    if out is None:
        with _made_on(stream):
            out = {"out": torch.empty((rows, Hq, D), dtype=dtype, device=q.device),
                   "status": torch.empty(B, dtype=torch.int32, device=q.device)}
    rc = (_lib or lib()).spec_prompt_attention(_PROMPT.pack(
        B, Hq, Hkv, D, code, window, sinks, scale, rows, cu, qp, kp, vp, qs, ks, vs,
        _on(out["out"], "out", device, dtype, shape), _on(out["status"], "status", device, _I32, (B,))), _raw_stream(stream, device))
    if rc != 0:
        _check(rc)
    return out


def spec_prompt_mark_timeout(marked=False, stream=None):
    """Clears what a wait of spec_prompt_attention that gave up has left on the current device; or sets it (True), so that the calls
    behind this one in the stream report TIMEOUT and a program's handling of that can be tried."""
    torch = _T or _cache_torch()
    _check((_lib or lib()).spec_prompt_mark_timeout(int(marked), _raw_stream(stream, torch.cuda.current_device())))


class RotaryTable:
    """The frequencies of rotary positions over the first ``dim`` elements of a head, on the device.

    Pair j of dim / 2 turns by base^(-2 j / dim) radians a position; ``scaling`` stretches that for contexts ``factor``
    times as long: "none", "linear" (position interpolation), "ntk" (a larger base), "yarn" (pairs that turn fewer than
    ``slow`` times in the ``original`` context are stretched, those that turn more than ``fast`` times are not, and between them
    the ramp is linear in the number of turns, as in the method's paper; models that were tuned with a ramp over the pairs'
    indices, or with another scaling, give their ``frequencies``).
    ``frequencies`` gives them (dim / 2 numbers, radians a position) instead, as they are: no scaling stretches them.  ``magnitude``
    multiplies what is turned (None: 0.1 ln(factor) + 1 for "yarn", of given frequencies too, otherwise 1).  A pair is (j, j + dim / 2), or with ``interleaved`` (2 j, 2 j + 1)."""

    SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

    def __init__(self, dim, base=10000.0, scaling="none", factor=1.0, original=4096, slow=1.0, fast=32.0, interleaved=False,
                 magnitude=None, frequencies=None, device="cuda"):
        torch = _T or _cache_torch()
        if scaling not in self.SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(self.SCALINGS)}, got {scaling!r}")
        if dim < 2 or dim % 2 != 0:
            raise ValueError(f"dim must be even and at least 2, got {dim}")
        n = dim // 2
        freq, mag = (ctypes.c_double * n)(), ctypes.c_float(1.0)
        if frequencies is None or (scaling == "yarn" and magnitude is None):
            _check(lib().spec_rotary_frequencies(dim, base, self.SCALINGS[scaling], factor, original, slow, fast, freq, ctypes.byref(mag)))
        if frequencies is not None:
            if len(frequencies) != n:
                raise ValueError(f"frequencies must be {n} numbers")
            freq[:] = [float(f) for f in frequencies]
        turns = (ctypes.c_int64 * n)()
        _check(lib().spec_rotary_turns(freq, n, turns))
        self.dim, self.interleaved = dim, bool(interleaved)
        self.magnitude = float(mag.value if magnitude is None else magnitude)
        self.frequencies = list(freq)
        self.turns = torch.tensor(list(turns), dtype=torch.int64).to(device)
        self._device, self._ptr = self.turns.get_device(), self.turns.data_ptr()

    def _on(self, device):
        if self._device != device:
            raise ValueError("the rotary table is on another device")
        return self._ptr


def spec_rotate(x, positions, rotary, out=None, stream=None):
    """x [rows, heads, D] (float32/bf16; rows may be slices of a wider projection) with every row turned by its position
    (positions [rows] int32).  Queries and keys that lie beside each other are one call.  ``out`` [rows, heads, D] may be
    such a slice too, or x itself.  Returns ``out``."""
    torch = _T or _cache_torch()
    shape, device, dtype = x.shape, x.get_device(), x.dtype
    if device < 0:
        raise TypeError("x must be a CUDA tensor")
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    if len(shape) != 3:
        raise ValueError("x must be [rows, heads, D]")
    rows, heads, D = shape
    xp, xs, _ = _packed(x, "x", device, dtype, heads, D)
    if out is None:
        with _made_on(stream):
            out = torch.empty(shape, dtype=dtype, device=x.device)
    op, os_ = _rows_into(out, "out", device, dtype, rows, heads, D)
    rc = (_lib or lib()).spec_rotate(_ROTATE.pack(
        heads, D, rotary.dim, rotary.interleaved, code, rotary.magnitude, rows, rotary._on(device),
        _on(positions, "positions", device, _I32, (rows,)), xp, xs, op, os_), _raw_stream(stream, device))
    if rc != 0:
        _check(rc)
    return out


def spec_cache_append_rotated(q, k, v, k_pages, v_pages, page_table, length, rotary, cu_rows=None, cu_drafts=None, kmax=None,
                              keep_keys=False, out=None, stream=None, reserved=None):
    """spec_cache_append with rotary positions on the way, for blocks and for whole prompts.

    Row i of stream b stands at position length[b] + i: its key goes turned, its value as it is, into one layer's pages, and its
    queries turned to out["q"]; with ``keep_keys`` the turned key goes to out["k"] as well (for spec_prompt_attention).  q [rows, Hq, D]
    (None: keys and values alone), k and v [rows, Hkv, D] may be slices of a wider projection.  The rows are packed by ``cu_rows`` [B + 1] int32 (their
    prefix sum; streams without rows are fine), or as verify blocks by ``cu_drafts`` [B + 1] (one row more than drafts; None: ``kmax``
    drafts each, where ``kmax`` is given: the most drafts of a stream).  ``reserved`` as in spec_cache_append.  Returns (and reuses) ``out``
    with q, k (None without), status [B]; out["q"] may be q itself, and out["k"] k."""
    torch = _T or _cache_torch()
    device, code, kpp, vpp, (num_pages, Hkv, page_size, D) = _layer_of(k_pages, v_pages)
    dtype = k_pages.dtype
    nk, ks, rows = _packed(k, "k", device, dtype, Hkv, D)
    nv, vs, v_rows = _packed(v, "v", device, dtype, Hkv, D)
    Hq = nq = qs = 0
    q_rows = rows
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [rows, Hq, D]")
        Hq = q.size(1)
        nq, qs, q_rows = _packed(q, "q", device, dtype, Hq, D)
    if v_rows != rows or q_rows != rows:
        raise ValueError("q, k and v must have the same rows")
    shape = page_table.shape
    if len(shape) != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B = shape[0]
    if cu_rows is not None:
        if cu_drafts is not None or kmax is not None:
            raise ValueError("cu_rows or cu_drafts and kmax, not both")
        cu, most, extra = _on(cu_rows, "cu_rows", device, _I32, (B + 1,)), rows, 0
    elif kmax is None:
        raise ValueError("cu_rows, or kmax (and cu_drafts), say how the rows are packed")
    else:
        most, extra = kmax + 1, 1
        if cu_drafts is None:
            cu = 0
            if rows != B * most:
                raise ValueError("without cu_drafts there are B * (kmax + 1) rows")
        else:
            cu = _on(cu_drafts, "cu_drafts", device, _I32, (B + 1,))
    if out is None:
        with _made_on(stream):
            out = {"q": None if q is None else torch.empty(q.shape, dtype=dtype, device=q.device),
                   "k": torch.empty(k.shape, dtype=dtype, device=k.device) if keep_keys else None,
                   "status": torch.empty(B, dtype=torch.int32, device=k.device)}
    oq = oqs = ok = oks = 0
    if q is not None:
        oq, oqs = _rows_into(out["q"], "out['q']", device, dtype, rows, Hq, D)
    if keep_keys:
        ok, oks = _rows_into(out["k"], "out['k']", device, dtype, rows, Hkv, D)
    rc = (_lib or lib()).spec_cache_append_rotated(_APPEND_ROTATED.pack(
        B, most, extra, Hq, Hkv, D, page_size, num_pages, shape[1], code, rotary.dim, rotary.interleaved, rotary.magnitude,
        rotary._on(device), cu, _on(length, "length", device, _I32, (B,)), _on(page_table, "page_table", device, _I32, shape),
        0 if reserved is None else _on(reserved, "reserved", device, _I32, (B,)), nq, nk, nv, qs, ks, vs, rows, oq, ok, oqs, oks,
        kpp, vpp, _on(out["status"], "status", device, _I32, (B,))), _raw_stream(stream, device))
    if rc != 0:
        _check(rc)
    return out
