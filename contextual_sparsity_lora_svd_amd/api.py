"""ctypes binding of libsparselora.so (argument marshalling only).

Every step of the computation runs in the library's HIP kernels; this module
allocates outputs and scratch with torch, passes raw device pointers and the
current HIP stream, and turns status codes into exceptions.  It never falls
back to any other implementation: if the library is missing it raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Dict, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsparselora.so")

SL_F32, SL_BF16 = 0, 1
SL_CRIT_SWIGLU_L2, SL_CRIT_L2, SL_CRIT_QK_NORM = 0, 1, 2
SL_MAX_SEQS = 64
SL_EST_MAXJOBS = 3

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t


class SlLayout(ctypes.Structure):
    _fields_ = [("batch", _i32), ("seq_len", _i32), ("ctx_len", ctypes.POINTER(_i32))]


class SlHeads(ctypes.Structure):
    _fields_ = [("n_q_heads", _i32), ("n_kv_heads", _i32), ("head_dim", _i32)]


class SlEstJob(ctypes.Structure):
    _fields_ = [("crit", ctypes.c_int), ("heads", SlHeads), ("Pt0", _vp), ("Q0", _vp), ("Pt1", _vp),
                ("Q1", _vp), ("N", _i64), ("k", _i32), ("idx", _vp), ("scores", _vp)]


class SlFfnWeights(ctypes.Structure):
    _fields_ = [("d_model", _i64), ("d_ff", _i64), ("lora_rank", _i32), ("lora_scale", ctypes.c_float),
                ("Wg", _vp), ("Wu", _vp), ("WdT", _vp), ("Ag", _vp), ("Bg", _vp), ("Au", _vp),
                ("Bu", _vp), ("Ad", _vp), ("Bd", _vp),
                ("Wg_q", _vp), ("Wu_q", _vp), ("WdT_q", _vp), ("Wg_s", _vp), ("Wu_s", _vp), ("WdT_s", _vp)]


class SlFfnGrads(ctypes.Structure):
    _fields_ = [("dAg", _vp), ("dBg", _vp), ("dAu", _vp), ("dBu", _vp), ("dAd", _vp), ("dBd", _vp)]


class SlQkvoWeights(ctypes.Structure):
    _fields_ = [("d_model", _i64), ("heads", SlHeads), ("lora_rank", _i32),
                ("lora_scale", ctypes.c_float),
                ("Wq", _vp), ("Wk", _vp), ("Wv", _vp), ("WoT", _vp),
                ("Aq", _vp), ("Bq", _vp), ("Ak", _vp), ("Bk", _vp), ("Av", _vp), ("Bv", _vp),
                ("Ao", _vp), ("Bo", _vp),
                ("Wq_q", _vp), ("Wk_q", _vp), ("Wv_q", _vp), ("WoT_q", _vp),
                ("Wq_s", _vp), ("Wk_s", _vp), ("Wv_s", _vp), ("WoT_s", _vp)]


class SlQkvoGrads(ctypes.Structure):
    _fields_ = [("dAq", _vp), ("dBq", _vp), ("dAk", _vp), ("dBk", _vp), ("dAv", _vp), ("dBv", _vp),
                ("dAo", _vp), ("dBo", _vp)]


class SlRotarySpec(ctypes.Structure):
    _fields_ = [("rot_dim", _i32), ("scaling", ctypes.c_int), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("original_len", _i64), ("low_turns", ctypes.c_double),
                ("high_turns", ctypes.c_double)]


class SlRotary(ctypes.Structure):
    _fields_ = [("rot_dim", _i32), ("interleaved", _i32), ("amplitude", ctypes.c_float), ("turns", _vp),
                ("pos", _vp)]


class SlDiffAttn(ctypes.Structure):
    _fields_ = [("heads", SlHeads), ("lambda_init", ctypes.c_float), ("scale", ctypes.c_float),
                ("causal", _i32), ("lens", ctypes.POINTER(_i32)), ("lq1", _vp), ("lk1", _vp), ("lq2", _vp),
                ("lk2", _vp)]


class SlDiffAttnGrads(ctypes.Structure):
    _fields_ = [("dlq1", _vp), ("dlk1", _vp), ("dlq2", _vp), ("dlk2", _vp)]


# name -> (restype, argtypes)
SIGNATURES = {
    "sl_abi_version": (ctypes.c_int, []),
    "sl_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "sl_last_error": (ctypes.c_char_p, []),
    "sl_estimator_workspace_bytes": (_sz, [_i64, _i64, _i32]),
    "sl_build_estimator": (ctypes.c_int, [ctypes.c_int, _vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp,
                                          _vp, _sz, _vp]),
    "sl_estimate_select_workspace_bytes": (_sz, [ctypes.c_int, ctypes.POINTER(SlLayout),
                                                 ctypes.POINTER(SlHeads), _i64, _i32, _i64]),
    "sl_estimate_select": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.POINTER(SlLayout),
                                          ctypes.POINTER(SlHeads), _vp, _i64, _i32, _vp, _vp, _vp,
                                          _vp, _i64, _i32, _vp, _vp, _vp, _sz, _vp]),
    "sl_estimate_select_noalloc": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.POINTER(SlLayout),
                                                  ctypes.POINTER(SlHeads), _vp, _i64, _i32, _vp, _vp, _vp,
                                                  _vp, _i64, _i32, _vp, _vp, _vp]),
    "sl_estimate_select_multi_workspace_bytes": (_sz, [ctypes.POINTER(SlLayout), _i64, _i32, _i32,
                                                       ctypes.POINTER(SlEstJob)]),
    "sl_estimate_select_multi": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(SlLayout), _vp, _i64, _i32,
                                                _i32, ctypes.POINTER(SlEstJob), _vp, _sz, _vp]),
    "sl_ffn_saved_bytes": (_sz, [ctypes.c_int, ctypes.POINTER(SlLayout), _i64, _i64, _i32, _i32]),
    "sl_ffn_workspace_bytes": (_sz, [ctypes.c_int, ctypes.POINTER(SlLayout), _i64, _i64, _i32,
                                     _i32]),
    "sl_ffn_fwd": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(SlLayout),
                                  ctypes.POINTER(SlFfnWeights), _vp, _i32, _vp, _vp, _vp, _sz, _vp,
                                  _sz, _vp]),
    "sl_ffn_bwd": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(SlLayout),
                                  ctypes.POINTER(SlFfnWeights), _vp, _i32, _vp, _vp, _sz, _vp, _vp,
                                  ctypes.POINTER(SlFfnGrads), _vp, _sz, _vp]),
    "sl_timer_enable": (ctypes.c_int, [ctypes.c_int]),
    "sl_gemm_config": (ctypes.c_int, [ctypes.c_int]),
    "sl_quantize_q4": (ctypes.c_int, [ctypes.c_int, _vp, _i64, _i64, _vp, _vp, _vp]),
    "sl_timer_select": (None, [ctypes.c_uint32]),
    "sl_timer_reset": (None, []),
    "sl_timer_read": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_int)]),
    "sl_qkvo_saved_bytes": (_sz, [ctypes.c_int, ctypes.POINTER(SlLayout),
                                  ctypes.POINTER(SlQkvoWeights)]),
    "sl_qkvo_workspace_bytes": (_sz, [ctypes.c_int, ctypes.POINTER(SlLayout),
                                      ctypes.POINTER(SlQkvoWeights), _i32, _i32]),
    "sl_qkvo_fwd": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(SlLayout),
                                   ctypes.POINTER(SlQkvoWeights), _vp, _vp, _i32, _vp, _i32, _vp,
                                   _vp, _vp, _vp, _vp, _vp, _sz, _vp, _sz, _vp]),
    "sl_qkvo_bwd": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(SlLayout),
                                   ctypes.POINTER(SlQkvoWeights), _vp, _vp, _i32, _vp, _i32, _vp,
                                   _vp, _sz, _vp, _vp, _vp, _vp, _vp, _vp,
                                   ctypes.POINTER(SlQkvoGrads), _vp, _sz, _vp]),
    "sl_rotary_table": (ctypes.c_int, [ctypes.POINTER(SlRotarySpec), ctypes.POINTER(ctypes.c_uint64),
                                       ctypes.POINTER(ctypes.c_float)]),
    "sl_rotary_apply": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(SlLayout), ctypes.POINTER(SlHeads),
                                       ctypes.POINTER(SlRotary), _vp, _vp, _vp, _vp, _i32, _vp]),
    "sl_head_norm_fwd": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(SlLayout), ctypes.POINTER(SlHeads),
                                        ctypes.POINTER(SlRotary), ctypes.c_float, _vp, _vp, _vp, _vp, _vp,
                                        _vp, _vp]),
    "sl_head_norm_workspace_bytes": (_sz, [ctypes.POINTER(SlLayout), ctypes.POINTER(SlHeads)]),
    "sl_head_norm_bwd": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(SlLayout), ctypes.POINTER(SlHeads),
                                        ctypes.POINTER(SlRotary), ctypes.c_float, _vp, _vp, _vp, _vp, _vp,
                                        _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sl_diff_attn_saved_bytes": (_sz, [ctypes.c_int, ctypes.POINTER(SlLayout), ctypes.POINTER(SlHeads)]),
    "sl_diff_attn_workspace_bytes": (_sz, [ctypes.c_int, ctypes.POINTER(SlLayout), ctypes.POINTER(SlHeads)]),
    "sl_diff_attn_fwd": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(SlLayout), ctypes.POINTER(SlDiffAttn),
                                        _vp, _vp, _vp, _vp, _vp, _sz, _vp, _sz, _vp]),
    "sl_diff_attn_bwd": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(SlLayout), ctypes.POINTER(SlDiffAttn),
                                        _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp, _vp, _vp,
                                        ctypes.POINTER(SlDiffAttnGrads), _vp, _sz, _vp]),
}

_lib = None


class SparseLoraError(RuntimeError):
    pass


def lib() -> ctypes.CDLL:
    """Load the HIP library; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise SparseLoraError(
                f"{LIB_PATH} is missing: build it with contextual_sparsity_lora_svd_amd.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int, what: str):
    if status != 0:
        L = lib()
        raise SparseLoraError(f"{what}: {L.sl_status_string(status).decode()} "
                              f"(status {status}): {L.sl_last_error().decode()}")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SL_BF16
    if t.dtype == torch.float32:
        return SL_F32
    raise SparseLoraError(f"unsupported dtype {t.dtype}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise SparseLoraError("tensors must be contiguous")
    return t.data_ptr()


def _stream() -> int:
    # torch.cuda.current_stream().cuda_stream without the Stream object (2.5 us)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


class Layout:
    """Host-side sequence layout (batch, seq_len, ctx_len[b])."""

    def __init__(self, ctx_len: Sequence[int], seq_len: int):
        self.ctx = (_i32 * len(ctx_len))(*[int(c) for c in ctx_len])
        self.c = SlLayout(len(ctx_len), int(seq_len), self.ctx)
        self.batch = len(ctx_len)
        self.seq_len = int(seq_len)

    @property
    def ref(self):
        return ctypes.byref(self.c)


def _bytes_tensor(n: int, device) -> torch.Tensor:
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device=device)


def k_from_ratio(n: int, sparsity_pct: int) -> int:
    """Channels kept at a per-layer sparsity percentage: round half up of
    (100 - p) * n / 100, at least 1."""
    return max((n * (100 - int(sparsity_pct)) + 50) // 100, 1)


TIMER_SLOTS = {"estimate": 0, "select": 1, "gu_fwd": 2, "down_fwd": 3, "dh_bwd": 4, "dx_bwd": 5,
               "qkv_fwd": 6, "o_fwd": 7, "da_bwd": 8, "dxqkv_bwd": 9}


def timer_enable(max_launches: int):
    _check(lib().sl_timer_enable(int(max_launches)), "sl_timer_enable")


def timer_select(slots):
    """Record only the named slots (None: all)."""
    mask = 0xFFFFFFFF if slots is None else sum(1 << TIMER_SLOTS[n] for n in slots)
    lib().sl_timer_select(mask)


def timer_reset():
    lib().sl_timer_reset()


def quantize_q4(W: torch.Tensor):
    """4-bit codes (uint8 [rows, cols / 2]) and block scales (fp32 [rows, cols / 64])
    of a frozen weight W [rows, cols], for FFNWeights' quantized base."""
    rows, cols = W.shape
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=W.device)
    scales = torch.empty((rows, max(cols // 64, 1)), dtype=torch.float32, device=W.device)
    _check(lib().sl_quantize_q4(_dtype_code(W), _ptr(W), rows, cols, _ptr(codes), _ptr(scales), _stream()),
           "sl_quantize_q4")
    return codes, scales


GEMM_WIDE, GEMM_TALL, GEMM_TALL_ALWAYS = 1, 2, 4


def gemm_config(variants: int = -1) -> int:
    """GEMM tile variants the calling thread allows, a bit mask: GEMM_WIDE
    (128 x 512 N-gather), GEMM_TALL (256 x 256 K-gather), GEMM_TALL_ALWAYS
    (tall tiles whatever their grid); 0 = 128 x 256 only; -1 only reads.
    Returns the previous setting."""
    return int(lib().sl_gemm_config(int(variants)))


def timer_read(slot: str):
    """(total milliseconds, launches) recorded for a slot since the last reset."""
    t = ctypes.c_double(0)
    n = ctypes.c_int(0)
    _check(lib().sl_timer_read(TIMER_SLOTS[slot], ctypes.byref(t), ctypes.byref(n)), "sl_timer_read")
    return t.value, n.value


# ---------------------------------------------------------------------------
def build_estimator(W: torch.Tensor, rank: int, iters: int = 0):
    """Truncated-SVD factors of a frozen weight W [out, in]: Pt [rank, in],
    Q [rank, out], sigma [rank] (fp32)."""
    L = lib()
    out_f, in_f = W.shape
    Pt = torch.empty(rank, in_f, dtype=W.dtype, device=W.device)
    Q = torch.empty(rank, out_f, dtype=W.dtype, device=W.device)
    sig = torch.empty(rank, dtype=torch.float32, device=W.device)
    ws = _bytes_tensor(L.sl_estimator_workspace_bytes(out_f, in_f, rank), W.device)
    _check(L.sl_build_estimator(_dtype_code(W), _ptr(W), out_f, in_f, rank, iters, _ptr(Pt),
                                _ptr(Q), _ptr(sig), _ptr(ws), ws.numel(), _stream()),
           "sl_build_estimator")
    return Pt, Q, sig


class EstimateBuffers:
    """Reusable idx / scores / scratch buffers of estimate_select."""

    def __init__(self, crit: int, layout: Layout, d_in: int, rank: int, N: int, k: int, device,
                 heads: Optional[Sequence[int]] = None, want_scores: bool = False):
        L = lib()
        self.heads = SlHeads(*heads) if heads is not None else None
        href = ctypes.byref(self.heads) if self.heads is not None else None
        self.idx = torch.empty(layout.batch, k, dtype=torch.int32, device=device)
        self.scores = (torch.empty(layout.batch, N, dtype=torch.float32, device=device)
                       if want_scores else None)
        self.ws = _bytes_tensor(L.sl_estimate_select_workspace_bytes(crit, layout.ref, href, d_in,
                                                                     rank, N), device)


def estimate_select(crit: int, X: torch.Tensor, layout: Layout, rank: int, Pt0, Q0, Pt1, Q1,
                    N: int, k: int, heads: Optional[Sequence[int]] = None,
                    want_scores: bool = False, bufs: Optional[EstimateBuffers] = None):
    """Per-sequence channel sets idx [batch, k] (int32, ascending) and,
    optionally, the scores [batch, N] (fp32)."""
    L = lib()
    bufs = bufs or EstimateBuffers(crit, layout, X.shape[1], rank, N, k, X.device, heads,
                                   want_scores)
    href = ctypes.byref(bufs.heads) if bufs.heads is not None else None
    _check(L.sl_estimate_select(crit, _dtype_code(X), layout.ref, href, _ptr(X), X.shape[1], rank,
                                _ptr(Pt0), _ptr(Q0), _ptr(Pt1), _ptr(Q1), N, k, _ptr(bufs.idx),
                                _ptr(bufs.scores), _ptr(bufs.ws), bufs.ws.numel(), _stream()),
           "sl_estimate_select")
    return bufs.idx, bufs.scores


def estimate_select_noalloc(crit: int, X: torch.Tensor, layout: Layout, rank: int, Pt0, Q0, Pt1, Q1,
                            N: int, k: int, idx: torch.Tensor, scores: Optional[torch.Tensor] = None,
                            heads: Optional[Sequence[int]] = None):
    """estimate_select into caller-owned idx [batch, k] (int32) and optional
    scores [batch, N] (fp32), with the library's fixed per-device scratch in
    place of a workspace: the call allocates no device memory."""
    L = lib()
    h = SlHeads(*heads) if heads is not None else None
    _check(L.sl_estimate_select_noalloc(crit, _dtype_code(X), layout.ref, ctypes.byref(h) if h else None,
                                        _ptr(X), X.shape[1], rank, _ptr(Pt0), _ptr(Q0), _ptr(Pt1), _ptr(Q1),
                                        N, k, _ptr(idx), _ptr(scores), _stream()),
           "sl_estimate_select_noalloc")
    return idx, scores


class EstimateMultiBuffers:
    """Reusable idx / scores / scratch buffers of estimate_select_multi.  Each
    job is a dict with crit, N, k and optionally heads and want_scores."""

    def __init__(self, layout: Layout, d_in: int, rank: int, jobs: Sequence[dict], device):
        L = lib()
        if not 1 <= len(jobs) <= SL_EST_MAXJOBS:
            raise ValueError(f"1..{SL_EST_MAXJOBS} jobs")
        self.c = (SlEstJob * len(jobs))()
        self.idx, self.scores = [], []
        for j, job in enumerate(jobs):
            c = self.c[j]
            c.crit, c.N, c.k = job["crit"], job["N"], job["k"]
            if job.get("heads") is not None:
                c.heads = SlHeads(*job["heads"])
            self.idx.append(torch.empty(layout.batch, job["k"], dtype=torch.int32, device=device))
            self.scores.append(torch.empty(layout.batch, job["N"], dtype=torch.float32, device=device)
                               if job.get("want_scores") else None)
        self.ws = _bytes_tensor(L.sl_estimate_select_multi_workspace_bytes(layout.ref, d_in, rank, len(jobs),
                                                                           self.c), device)


def estimate_select_multi(X: torch.Tensor, layout: Layout, rank: int, jobs: Sequence[dict],
                          bufs: Optional[EstimateMultiBuffers] = None):
    """Several criteria over one input X in one call.  Each job is a dict with
    crit, Pt0, Q0 (and Pt1, Q1 unless L2), N, k and optionally heads (QK-norm)
    and want_scores.  Returns [(idx, scores)] in job order, as separate
    estimate_select calls would."""
    L = lib()
    bufs = bufs or EstimateMultiBuffers(layout, X.shape[1], rank, jobs, X.device)
    for j, job in enumerate(jobs):
        c = bufs.c[j]
        c.Pt0, c.Q0 = _ptr(job["Pt0"]), _ptr(job["Q0"])
        c.Pt1, c.Q1 = _ptr(job.get("Pt1")), _ptr(job.get("Q1"))
        c.idx, c.scores = _ptr(bufs.idx[j]), _ptr(bufs.scores[j])
    _check(L.sl_estimate_select_multi(_dtype_code(X), layout.ref, _ptr(X), X.shape[1], rank, len(jobs), bufs.c,
                                      _ptr(bufs.ws), bufs.ws.numel(), _stream()),
           "sl_estimate_select_multi")
    return list(zip(bufs.idx, bufs.scores))


class FFNWeights:
    """Device tensors of one FFN layer: Wg, Wu, WdT, Ag, Bg, Au, Bu, Ad, Bd.

    A 4-bit frozen base replaces Wg, Wu, WdT by Wg_q, Wu_q, WdT_q (uint8 codes
    [d_ff, d_model / 2]) and Wg_s, Wu_s, WdT_s (fp32 scales [d_ff, d_model / 64])."""

    NAMES = ("Wg", "Wu", "WdT", "Ag", "Bg", "Au", "Bu", "Ad", "Bd")
    QNAMES = ("Wg_q", "Wu_q", "WdT_q", "Wg_s", "Wu_s", "WdT_s")

    def __init__(self, t: Dict[str, torch.Tensor], lora_scale: float = 1.0):
        self.t = t
        self.quantized = "Wg_q" in t
        if self.quantized:
            d_ff, half = t["Wg_q"].shape
            d_model = 2 * half
        else:
            d_ff, d_model = t["Wg"].shape
        r = t["Ag"].shape[0]
        self.c = SlFfnWeights(d_model, d_ff, r, float(lora_scale),
                              *[_ptr(t[n]) if n in t else None for n in self.NAMES + self.QNAMES])
        self.d_model, self.d_ff, self.r = d_model, d_ff, r
        self.dtype = _dtype_code(t["Ag"])

    @property
    def ref(self):
        return ctypes.byref(self.c)


class FFNWorkspace:
    """Reusable saved + scratch buffers for one (layout, shape, k)."""

    def __init__(self, w: FFNWeights, layout: Layout, k: int, device):
        L = lib()
        self.saved = _bytes_tensor(L.sl_ffn_saved_bytes(w.dtype, layout.ref, w.d_model, w.d_ff, w.r, k),
                                   device)
        self.ws = _bytes_tensor(L.sl_ffn_workspace_bytes(w.dtype, layout.ref, w.d_model, w.d_ff, w.r, k),
                                device)


def ffn_fwd(w: FFNWeights, X: torch.Tensor, layout: Layout, k: int, idx: torch.Tensor,
            buf: Optional[FFNWorkspace] = None, Y: Optional[torch.Tensor] = None):
    L = lib()
    buf = buf or FFNWorkspace(w, layout, k, X.device)
    Y = Y if Y is not None else torch.empty_like(X)
    _check(L.sl_ffn_fwd(w.dtype, layout.ref, w.ref, _ptr(X), k, _ptr(idx), _ptr(Y),
                        _ptr(buf.saved), buf.saved.numel(), _ptr(buf.ws), buf.ws.numel(), _stream()),
           "sl_ffn_fwd")
    return Y, buf


def ffn_bwd(w: FFNWeights, X: torch.Tensor, layout: Layout, k: int, idx: torch.Tensor,
            buf: FFNWorkspace, dY: torch.Tensor, out: Optional[Dict[str, torch.Tensor]] = None):
    L = lib()
    dev = X.device
    if out is None:
        out = {"dX": torch.empty_like(X)}
        for n in ("Ag", "Bg", "Au", "Bu", "Ad", "Bd"):
            out["d" + n] = torch.empty(w.t[n].shape, dtype=torch.float32, device=dev)
    g = SlFfnGrads(*[_ptr(out[n]) for n in ("dAg", "dBg", "dAu", "dBu", "dAd", "dBd")])
    _check(L.sl_ffn_bwd(w.dtype, layout.ref, w.ref, _ptr(X), k, _ptr(idx), _ptr(buf.saved),
                        buf.saved.numel(), _ptr(dY), _ptr(out["dX"]), ctypes.byref(g), _ptr(buf.ws),
                        buf.ws.numel(), _stream()),
           "sl_ffn_bwd")
    return out


class QKVOWeights:
    """Device tensors of one attention block's projections.  A 4-bit frozen
    base replaces Wq, Wk, Wv by Wq_q, Wk_q, Wv_q with Wq_s, Wk_s, Wv_s, and WoT
    by WoT_q with WoT_s (the format of FFNWeights' quantized base)."""

    NAMES = ("Wq", "Wk", "Wv", "WoT", "Aq", "Bq", "Ak", "Bk", "Av", "Bv", "Ao", "Bo")
    QNAMES = ("Wq_q", "Wk_q", "Wv_q", "WoT_q", "Wq_s", "Wk_s", "Wv_s", "WoT_s")

    def __init__(self, t: Dict[str, torch.Tensor], heads: Sequence[int], lora_scale: float = 1.0):
        self.t = t
        self.heads = tuple(int(h) for h in heads)
        d_model = t["Aq"].shape[1]
        r = t["Aq"].shape[0]
        self.c = SlQkvoWeights(d_model, SlHeads(*self.heads), r, float(lora_scale),
                               *[_ptr(t[n]) if n in t else None for n in self.NAMES + self.QNAMES])
        self.d_model, self.r = d_model, r
        self.dtype = _dtype_code(t["Aq"])

    @property
    def ref(self):
        return ctypes.byref(self.c)


class QKVOWorkspace:
    def __init__(self, w: QKVOWeights, layout: Layout, k_qk: int, k_vo: int, device):
        L = lib()
        self.saved = _bytes_tensor(L.sl_qkvo_saved_bytes(w.dtype, layout.ref, w.ref), device)
        self.ws = _bytes_tensor(L.sl_qkvo_workspace_bytes(w.dtype, layout.ref, w.ref, k_qk, k_vo),
                                device)


def qkvo_fwd(w: QKVOWeights, X: Optional[torch.Tensor], a: Optional[torch.Tensor], layout: Layout,
             k_qk: int, idx_qk: torch.Tensor, k_vo: int, idx_vo: torch.Tensor,
             buf: Optional[QKVOWorkspace] = None, outs: Optional[Dict[str, torch.Tensor]] = None):
    L = lib()
    ref = X if X is not None else a
    dev = ref.device
    hq, hkv, hd = w.heads
    T = layout.batch * layout.seq_len
    buf = buf or QKVOWorkspace(w, layout, k_qk, k_vo, dev)
    outs = dict(outs or {})
    if X is not None:
        outs.setdefault("q", torch.empty(T, hq * hd, dtype=ref.dtype, device=dev))
        outs.setdefault("k", torch.empty(T, hkv * hd, dtype=ref.dtype, device=dev))
        outs.setdefault("v", torch.empty(T, hkv * hd, dtype=ref.dtype, device=dev))
    if a is not None:
        outs.setdefault("o", torch.empty(T, w.d_model, dtype=ref.dtype, device=dev))
    _check(L.sl_qkvo_fwd(w.dtype, layout.ref, w.ref, _ptr(X), _ptr(a), k_qk, _ptr(idx_qk), k_vo,
                         _ptr(idx_vo), _ptr(outs.get("q")), _ptr(outs.get("k")), _ptr(outs.get("v")),
                         _ptr(outs.get("o")), _ptr(buf.saved), buf.saved.numel(), _ptr(buf.ws),
                         buf.ws.numel(), _stream()),
           "sl_qkvo_fwd")
    return outs, buf


def qkvo_bwd(w: QKVOWeights, X: Optional[torch.Tensor], a: Optional[torch.Tensor], layout: Layout,
             k_qk: int, idx_qk: torch.Tensor, k_vo: int, idx_vo: torch.Tensor, buf: QKVOWorkspace,
             dq=None, dk=None, dv=None, d_out=None, out: Optional[Dict[str, torch.Tensor]] = None):
    L = lib()
    ref = X if X is not None else a
    dev = ref.device
    out = dict(out or {})
    if dq is not None:
        out.setdefault("dX", torch.empty_like(X))
        for n in ("Aq", "Bq", "Ak", "Bk", "Av", "Bv"):
            out.setdefault("d" + n, torch.empty(w.t[n].shape, dtype=torch.float32, device=dev))
    if d_out is not None:
        out.setdefault("da", torch.empty_like(a))
        for n in ("Ao", "Bo"):
            out.setdefault("d" + n, torch.empty(w.t[n].shape, dtype=torch.float32, device=dev))
    g = SlQkvoGrads(*[_ptr(out.get(n)) for n in ("dAq", "dBq", "dAk", "dBk", "dAv", "dBv", "dAo",
                                                  "dBo")])
    _check(L.sl_qkvo_bwd(w.dtype, layout.ref, w.ref, _ptr(X), _ptr(a), k_qk, _ptr(idx_qk), k_vo,
                         _ptr(idx_vo), _ptr(buf.saved), buf.saved.numel(), _ptr(dq), _ptr(dk),
                         _ptr(dv), _ptr(d_out), _ptr(out.get("dX")), _ptr(out.get("da")),
                         ctypes.byref(g), _ptr(buf.ws), buf.ws.numel(), _stream()),
           "sl_qkvo_bwd")
    return out


# ---------------------------------------------------------------------------
# Between the q/k/v and the o projection: rotary positions, head norms,
# differential attention.
def _check_rows(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, dev: Optional[int] = None) -> int:
    """The pointer of a contiguous tensor of this shape and type on the current
    device (``dev``, where the caller has it at hand)."""
    if t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.is_cuda:
        if t.get_device() == (torch.cuda.current_device() if dev is None else dev):
            return t.data_ptr()
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise SparseLoraError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise SparseLoraError(f"{name}: tensors must be contiguous")
    if not t.is_cuda:
        raise SparseLoraError(f"{name}: tensors must be on the GPU, got {t.device}")
    raise SparseLoraError(f"{name}: on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")


def _refuse_overlap(outs, ins, in_place=()):
    """Refuse outputs ((name, tensor) pairs, None left out) that share memory with each
    other or with an input, but the ``in_place`` pairs (output, input) of the same rows.
    Only outputs that a caller gives can."""
    span = lambda t: (t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
    outs = [(n, span(t)) for n, t in outs if t is not None]
    ins = [(n, span(t)) for n, t in ins if t is not None]
    for i, (n, o) in enumerate(outs):
        for m, x in outs[:i] + ins:
            if o[0] < x[1] and x[0] < o[1] and not (o == x and (n, m) in in_place):
                raise SparseLoraError(f"{n} and {m} may not share memory here")


def _current(t: torch.Tensor) -> Optional[int]:
    """The current device, where there is one to ask for."""
    return torch.cuda.current_device() if t.is_cuda else None


ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "wavelength": 3, "yarn": 4}


class Rotary:
    """The frequency table of rotary positions: pair i of a head's first
    ``rot_dim`` values turns by ``position * base**(-2 i / rot_dim)``, pairs
    being values i and i + rot_dim / 2, or 2 i and 2 i + 1 (``interleaved``).

    ``scaling`` stretches the positions by ``factor`` for long contexts:
    "linear" (every frequency), "base" (a larger base), "wavelength" (pairs
    that turn fewer than ``low_turns`` times within ``original_len``, none
    above ``high_turns``, linear between) or "yarn" (a ramp over the pair
    index, with the amplitude 0.1 ln(factor) + 1)."""

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, original_len: int = 4096, low_turns: float = 1.0,
                 high_turns: Optional[float] = None, device="cuda"):
        if scaling not in ROPE_SCALINGS:
            raise SparseLoraError(f"unknown rotary scaling {scaling!r}: one of {sorted(ROPE_SCALINGS)}")
        if high_turns is None:
            high_turns = 32.0 if scaling == "yarn" else 4.0
        spec = SlRotarySpec(int(rot_dim), ROPE_SCALINGS[scaling], float(base), float(factor), int(original_len),
                            float(low_turns), float(high_turns))
        table = (ctypes.c_uint64 * max(int(rot_dim) // 2, 1))()
        amp = ctypes.c_float(0)
        _check(lib().sl_rotary_table(ctypes.byref(spec), table, ctypes.byref(amp)), "sl_rotary_table")
        self.rot_dim, self.interleaved, self.amplitude = int(rot_dim), bool(interleaved), amp.value
        # torch holds the table's 64 bits as signed integers
        self.turns = torch.tensor([ctypes.c_int64(x).value for x in table], dtype=torch.int64).to(device)

    def _c(self, pos: Optional[torch.Tensor], T: int, dev: Optional[int]) -> SlRotary:
        pp = None if pos is None else _check_rows("pos", pos, (T,), torch.int32, dev)
        tp = _check_rows("turns", self.turns, (self.rot_dim // 2,), torch.int64, dev)
        return SlRotary(self.rot_dim, self.interleaved, self.amplitude, tp, pp)


def _check_scratch(name: str, ws: torch.Tensor, like: torch.Tensor) -> int:
    if ws.get_device() != like.get_device():
        raise SparseLoraError(f"{name}: buffers on {ws.device}, tensors on {like.device}")
    return _ptr(ws)


@functools.lru_cache(maxsize=64)
def _heads_ref(heads: tuple):
    """The C struct of (n_q_heads, n_kv_heads, head_dim); calls only read it."""
    h = SlHeads(*heads)
    return h, ctypes.byref(h)


def _pair_ptrs(names, q, k, T, heads, dtype, dev):
    """Pointers of a q-shaped and an optional k-shaped tensor."""
    hd = heads[2]
    qp = _check_rows(names[0], q, (T, heads[0] * hd), dtype, dev)
    kp = None if k is None else _check_rows(names[1], k, (T, heads[1] * hd), dtype, dev)
    return qp, kp


_IN_PLACE = (("q_out", "q"), ("k_out", "k"))


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], layout: Layout, heads: Sequence[int], rot: Rotary,
           pos: Optional[torch.Tensor] = None, inverse: bool = False,
           out: Optional[Sequence[Optional[torch.Tensor]]] = None):
    """(q, k) [T, H * head_dim] with the position rotation applied to every
    head; ``inverse`` turns back, which is the gradient.  ``pos`` [T] int32,
    or None: the row's place in its sequence.  ``out`` (for q, for k) may hold
    q and k themselves, each in its own place.  k may be None."""
    dt, T, dev = _dtype_code(q), layout.batch * layout.seq_len, _current(q)
    qp, kp = _pair_ptrs(("q", "k"), q, k, T, heads, q.dtype, dev)
    if out is None:
        qo, ko = torch.empty_like(q), None if k is None else torch.empty_like(k)
        qop, kop = qo.data_ptr(), None if k is None else ko.data_ptr()
    else:
        qo, ko = out
        if (k is None) != (ko is None):
            raise SparseLoraError("out must hold a tensor for each input")
        qop, kop = _pair_ptrs(("q_out", "k_out"), qo, ko, T, heads, q.dtype, dev)
        _refuse_overlap((("q_out", qo), ("k_out", ko)), (("q", q), ("k", k), ("pos", pos), ("turns", rot.turns)), _IN_PLACE)
    r = rot._c(pos, T, dev)
    _check(lib().sl_rotary_apply(dt, layout.ref, _heads_ref(tuple(heads))[1], ctypes.byref(r), qp, kp, qop, kop,
                                 int(inverse), _stream()), "sl_rotary_apply")
    return qo, ko


class HeadNormWorkspace:
    """Reusable scratch of head_norm_bwd."""

    def __init__(self, layout: Layout, heads: Sequence[int], device):
        self.ws = _bytes_tensor(lib().sl_head_norm_workspace_bytes(layout.ref, ctypes.byref(SlHeads(*heads))),
                                device)


def head_norm_fwd(q: torch.Tensor, k: Optional[torch.Tensor], wq: torch.Tensor, wk: Optional[torch.Tensor],
                  layout: Layout, heads: Sequence[int], rot: Optional[Rotary] = None,
                  pos: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  out: Optional[Sequence[Optional[torch.Tensor]]] = None):
    """(q, k) with every head divided by its root mean square and multiplied
    by wq / wk [head_dim] (fp32), then rotated (``rot`` None: not).  k and wk
    may both be None."""
    dt, T, dev, hd = _dtype_code(q), layout.batch * layout.seq_len, _current(q), heads[2]
    qp, kp = _pair_ptrs(("q", "k"), q, k, T, heads, q.dtype, dev)
    wqp = _check_rows("wq", wq, (hd,), torch.float32, dev)
    wkp = None if wk is None else _check_rows("wk", wk, (hd,), torch.float32, dev)
    if out is None:
        qo, ko = torch.empty_like(q), None if k is None else torch.empty_like(k)
        qop, kop = qo.data_ptr(), None if k is None else ko.data_ptr()
    else:
        qo, ko = out
        qop, kop = _pair_ptrs(("q_out", "k_out"), qo, ko, T, heads, q.dtype, dev)
        _refuse_overlap((("q_out", qo), ("k_out", ko)), (("q", q), ("k", k), ("wq", wq), ("wk", wk), ("pos", pos)), _IN_PLACE)
    r = ctypes.byref(rot._c(pos, T, dev)) if rot is not None else None
    _check(lib().sl_head_norm_fwd(dt, layout.ref, _heads_ref(tuple(heads))[1], r, eps, qp, kp, wqp, wkp, qop, kop,
                                  _stream()), "sl_head_norm_fwd")
    return qo, ko


def head_norm_bwd(q: torch.Tensor, k: Optional[torch.Tensor], wq: torch.Tensor, wk: Optional[torch.Tensor],
                  layout: Layout, heads: Sequence[int], dq_out: torch.Tensor, dk_out: Optional[torch.Tensor],
                  rot: Optional[Rotary] = None, pos: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  buf: Optional[HeadNormWorkspace] = None, out: Optional[Dict[str, torch.Tensor]] = None):
    """Gradients dq, dk (call dtype) and dwq, dwk (fp32) of head_norm_fwd; q
    and k are its inputs.  ``out`` may hold results to write into: dq may be
    dq_out or q, and dk dk_out or k."""
    dt, T, dev, hd = _dtype_code(q), layout.batch * layout.seq_len, _current(q), heads[2]
    qp, kp = _pair_ptrs(("q", "k"), q, k, T, heads, q.dtype, dev)
    gqp, gkp = _pair_ptrs(("dq_out", "dk_out"), dq_out, dk_out, T, heads, q.dtype, dev)
    wqp = _check_rows("wq", wq, (hd,), torch.float32, dev)
    wkp = None if wk is None else _check_rows("wk", wk, (hd,), torch.float32, dev)
    buf = buf or HeadNormWorkspace(layout, heads, q.device)
    given = bool(out)
    out = dict(out or {})
    for n, x, w in (("q", q, wq), ("k", k, wk)):
        if x is not None:
            if "d" + n not in out:
                out["d" + n] = torch.empty_like(x)
            if "dw" + n not in out:
                out["dw" + n] = torch.empty_like(w)
    dqp, dkp = _pair_ptrs(("dq", "dk"), out["dq"], out.get("dk"), T, heads, q.dtype, dev)
    dwq = _check_rows("dwq", out["dwq"], (hd,), torch.float32, dev)
    dwk = _check_rows("dwk", out["dwk"], (hd,), torch.float32, dev) if "dwk" in out else None
    if given:
        _refuse_overlap([(n, out.get(n)) for n in ("dq", "dk", "dwq", "dwk")],
                        (("q", q), ("k", k), ("wq", wq), ("wk", wk), ("dq_out", dq_out), ("dk_out", dk_out), ("pos", pos),
                         ("ws", buf.ws)), (("dq", "dq_out"), ("dk", "dk_out"), ("dq", "q"), ("dk", "k")))
    r = ctypes.byref(rot._c(pos, T, dev)) if rot is not None else None
    _check(lib().sl_head_norm_bwd(dt, layout.ref, _heads_ref(tuple(heads))[1], r, eps, qp, kp, wqp, wkp, gqp, gkp,
                                  dqp, dkp, dwq, dwk, _check_scratch("ws", buf.ws, q), buf.ws.numel(), _stream()),
           "sl_head_norm_bwd")
    return out


def pair_heads(heads: Sequence[int]):
    """The heads that the projections around differential attention of ``heads``
    take (QKVOWeights, and the heads of the QK-norm criterion): its pairs, each
    one head of twice the width, so that query head 2 h + m and the columns 2 h + m
    of a keep the channels of kv head 2 (h / (Hq / Hkv)) + m, which they meet."""
    hq, hkv, hd = (int(h) for h in heads)
    if hq % 2 or hkv % 2:
        raise SparseLoraError(f"differential heads come in pairs: {hq} query and {hkv} kv heads")
    return hq // 2, hkv // 2, 2 * hd


class DiffAttnParams:
    """Differential attention's learned vectors lq1, lk1, lq2, lk2 [head_dim]
    (fp32 device tensors; lambda = exp(lq1.lk1) - exp(lq2.lk2) + lambda_init)
    and its settings.  ``scale`` None: head_dim ** -0.5."""

    NAMES = ("lq1", "lk1", "lq2", "lk2")

    def __init__(self, t: Dict[str, torch.Tensor], heads: Sequence[int], lambda_init: float = 0.8,
                 scale: Optional[float] = None, causal: bool = True):
        self.t = t
        self.heads = tuple(int(h) for h in heads)
        self.lambda_init, self.causal = float(lambda_init), bool(causal)
        self.scale = float(scale) if scale is not None else float(max(self.heads[2], 1)) ** -0.5

    def _c(self, lens, dev: Optional[int]) -> SlDiffAttn:
        shape = (self.heads[2],)
        ptrs = [_check_rows(n, self.t[n], shape, torch.float32, dev) for n in self.NAMES]
        return SlDiffAttn(SlHeads(*self.heads), self.lambda_init, self.scale, int(self.causal), lens, *ptrs)


class DiffAttnWorkspace:
    """Saved and scratch buffers of one differential attention call and its
    backward, with the sequences' valid lengths (None: every row).  Only the
    backward needs scratch (``ws``); without ``scratch`` it is made where it is
    first asked for, by the first backward that gets these buffers."""

    def __init__(self, p: DiffAttnParams, layout: Layout, dtype: torch.dtype, device,
                 lens: Optional[Sequence[int]] = None, scratch: bool = True):
        L = lib()
        code = {torch.bfloat16: SL_BF16, torch.float32: SL_F32}.get(dtype)
        if code is None:
            raise SparseLoraError(f"unsupported dtype {dtype}")
        if lens is not None and len(lens) != layout.batch:
            raise SparseLoraError(f"lens holds {len(lens)} lengths for {layout.batch} sequences")
        self.lens = None if lens is None else (_i32 * len(lens))(*[int(n) for n in lens])
        self.made_for = (layout.batch, layout.seq_len, p.heads, dtype)
        h = SlHeads(*p.heads)
        self.saved = _bytes_tensor(L.sl_diff_attn_saved_bytes(code, layout.ref, ctypes.byref(h)), device)
        nbytes = L.sl_diff_attn_workspace_bytes(code, layout.ref, ctypes.byref(h))
        self._ws_bytes, self._ws = nbytes, _bytes_tensor(nbytes, device) if scratch else None

    @property
    def ws(self) -> torch.Tensor:
        if self._ws is None:
            self._ws = _bytes_tensor(self._ws_bytes, self.saved.device)
        return self._ws


def _diff_buffers(buf: DiffAttnWorkspace, p: DiffAttnParams, layout: Layout, q: torch.Tensor):
    """(saved, bytes, ws, bytes) of a call over q; no ws where none has been made."""
    if buf.made_for != (layout.batch, layout.seq_len, p.heads, q.dtype):
        raise SparseLoraError(f"buffers made for (batch, seq_len, heads, dtype) = {buf.made_for}, "
                              f"call of {(layout.batch, layout.seq_len, p.heads, q.dtype)}")
    ws = (None, 0) if buf._ws is None else (_check_scratch("ws", buf._ws, q), buf._ws.numel())
    return (_check_scratch("saved", buf.saved, q), buf.saved.numel(), *ws)


def diff_attn_fwd(p: DiffAttnParams, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, layout: Layout,
                  lens: Optional[Sequence[int]] = None, buf: Optional[DiffAttnWorkspace] = None,
                  out: Optional[torch.Tensor] = None):
    """a [T, Hq * head_dim] and the buffers its backward reads.  ``lens``
    [batch]: valid rows per sequence (a given ``buf`` holds its own)."""
    if k is None or v is None:
        raise SparseLoraError("q, k and v are required")
    dt, T, dev = _dtype_code(q), layout.batch * layout.seq_len, _current(q)
    qp, kp = _pair_ptrs(("q", "k"), q, k, T, p.heads, q.dtype, dev)
    vp = _check_rows("v", v, k.shape, q.dtype, dev)
    if buf is None:
        buf = DiffAttnWorkspace(p, layout, q.dtype, q.device, lens, scratch=False)
    elif lens is not None:
        raise SparseLoraError("lens belongs to the buffers: give it to DiffAttnWorkspace")
    a = out if out is not None else torch.empty_like(q)
    ap = _check_rows("a", a, q.shape, q.dtype, dev)
    saved, ns, ws, nw = _diff_buffers(buf, p, layout, q)
    if out is not None:
        _refuse_overlap((("a", a),), (("q", q), ("k", k), ("v", v), ("saved", buf.saved), *p.t.items()))
    c = p._c(buf.lens, dev)
    _check(lib().sl_diff_attn_fwd(dt, layout.ref, ctypes.byref(c), qp, kp, vp, ap, saved, ns, ws, nw, _stream()),
           "sl_diff_attn_fwd")
    return a, buf


def diff_attn_bwd(p: DiffAttnParams, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, a: torch.Tensor,
                  layout: Layout, buf: DiffAttnWorkspace, da: torch.Tensor,
                  out: Optional[Dict[str, torch.Tensor]] = None):
    """Gradients dq, dk, dv (call dtype) and dlq1, dlk1, dlq2, dlk2 (fp32); a
    and buf are diff_attn_fwd's."""
    if k is None or v is None:
        raise SparseLoraError("q, k and v are required")
    dt, T, dev = _dtype_code(q), layout.batch * layout.seq_len, _current(q)
    qp, kp = _pair_ptrs(("q", "k"), q, k, T, p.heads, q.dtype, dev)
    vp = _check_rows("v", v, k.shape, q.dtype, dev)
    ap = _check_rows("a", a, q.shape, q.dtype, dev)
    gp = _check_rows("da", da, q.shape, q.dtype, dev)
    given = bool(out)
    out = dict(out or {})
    for n, x in (("dq", q), ("dk", k), ("dv", v)):
        if n not in out:
            out[n] = torch.empty_like(x)
    for n in p.NAMES:
        if "d" + n not in out:
            out["d" + n] = torch.empty_like(p.t[n])
    dqp, dkp = _pair_ptrs(("dq", "dk"), out["dq"], out["dk"], T, p.heads, q.dtype, dev)
    dvp = _check_rows("dv", out["dv"], v.shape, q.dtype, dev)
    shape = (p.heads[2],)
    g = SlDiffAttnGrads(*[_check_rows("d" + n, out["d" + n], shape, torch.float32, dev) for n in p.NAMES])
    buf.ws                                       # made here, if not before
    saved, ns, ws, nw = _diff_buffers(buf, p, layout, q)
    if given:
        _refuse_overlap([(n, out[n]) for n in ("dq", "dk", "dv", *("d" + m for m in p.NAMES))],
                        (("q", q), ("k", k), ("v", v), ("a", a), ("da", da), ("saved", buf.saved), ("ws", buf.ws),
                         *p.t.items()))
    c = p._c(buf.lens, dev)
    _check(lib().sl_diff_attn_bwd(dt, layout.ref, ctypes.byref(c), qp, kp, vp, ap, saved, ns, gp, dqp, dkp, dvp,
                                  ctypes.byref(g), ws, nw, _stream()), "sl_diff_attn_bwd")
    return out
