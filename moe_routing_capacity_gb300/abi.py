"""ctypes binding of ``libmoe_pooled_wave.so`` (the C ABI in
``include/moe_pooled_wave.h``).

Argument marshalling only: each function takes torch tensors, checks dtype,
device and contiguity, and passes raw pointers, sizes and the current CUDA
stream to the C entry point of the same name.  Every step of the layer runs
in the library's kernels; if the library is missing this module raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_pooled_wave.so")

MOE_OK, MOE_EINVAL, MOE_ENOSPC, MOE_ECUDA, MOE_ETIMEOUT, MOE_ENODEV = 0, -1, -2, -3, -4, -5

# Every entry point the header declares (checked by the tests).
EXPORTS = ("moe_plan", "moe_router_topk", "moe_latent_proj", "moe_route_project", "moe_matmul",
           "moe_dispatch_pooled",
           "moe_dispatch_pooled_noalloc", "moe_expert_ffn_grouped", "moe_dispatch_expert_waves",
           "moe_dispatch_shared_overlap", "moe_balance_update", "moe_balance_update_window",
           "moe_plan_ragged", "moe_dispatch_ragged", "moe_dispatch_ragged_shared_overlap",
           "moe_expert_ffn_ragged",
           "moe_backward_plan", "moe_layer_backward", "moe_backward_plan_ragged",
           "moe_layer_backward_ragged", "moe_combine", "moe_trace_begin", "moe_trace_mark",
           "moe_trace_end", "moe_trace_event", "moe_check_status", "moe_strerror",
           "moe_abi_version", "moe_layer_forward", "moe_host_pipe_create", "moe_host_pipe_submit",
           "moe_host_pipe_sync", "moe_host_pipe_destroy",
           "moe_norm_residual", "moe_norm_residual_workspace", "moe_norm_residual_backward",
           "moe_rotary_make_table", "moe_rotary", "moe_attention_workspace",
           "moe_attention_plan", "moe_attention_forward", "moe_attention_backward",
           "moe_grad_clip_workspace", "moe_grad_clip",
           "moe_head_norm_rotary", "moe_head_norm_rotary_workspace",
           "moe_head_norm_rotary_backward", "moe_router_select", "moe_router_select_backward",
           "moe_route_logits", "moe_layer_backward_routed",
           "moe_embedding", "moe_embedding_workspace", "moe_embedding_plan",
           "moe_embedding_backward", "moe_distill_loss", "moe_distill_loss_backward")
# Declared in the header too, but exported by the checked build only.
CHECKED_ONLY = ("moe_check_set_wave_wait_limit_ns",)


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {code} ({strerror(code)})")
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d_model", ctypes.c_int32), ("d_latent", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("n_ranks", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("n_waves", ctypes.c_int32),
                ("n_shared", ctypes.c_int32), ("h_expert", ctypes.c_int32),
                ("h_shared", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("cf_send", ctypes.c_double), ("cf_recv", ctypes.c_double)]


class Plan(ctypes.Structure):
    _fields_ = [("tokens_per_rank", ctypes.c_int64), ("experts_per_rank", ctypes.c_int32),
                ("experts_per_wave", ctypes.c_int32), ("c_send", ctypes.c_int32),
                ("c_recv", ctypes.c_int32), ("pool_rows", ctypes.c_int64),
                ("pool_row_bytes", ctypes.c_int64), ("ws_dispatch_bytes", ctypes.c_int64),
                ("ws_ffn_bytes", ctypes.c_int64), ("h_offset_bytes", ctypes.c_int64)]


class DropStats(ctypes.Structure):
    _fields_ = [("assignments", ctypes.c_int64), ("kept", ctypes.c_int64),
                ("dropped_send", ctypes.c_int64), ("dropped_recv", ctypes.c_int64),
                ("max_send_fill", ctypes.c_int32), ("max_expert_rows", ctypes.c_int32),
                ("status", ctypes.c_int32), ("reserved", ctypes.c_int32)]


STATS_WORDS = ctypes.sizeof(DropStats) // 8    # int64 words of a stats record

BWD_WS_FIELDS = ("dc", "da", "dgs", "dus", "dw", "rowinv", "dxpool", "dh", "dg", "du", "xe", "dye",
                 "dz", "dlogits", "tiles", "hp", "poff", "total")


class BackwardWs(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in BWD_WS_FIELDS]


BWD_ARG_FIELDS = ("x", "Wr", "W_ld", "Wg", "Wu", "Wd", "W_lu", "Wsg", "Wsu", "Wsd", "idx", "w",
                  "pool", "slot_of", "expert_rows", "expert_count", "h", "ypool", "c", "a",
                  "dout", "dx", "dWr", "dW_ld", "dWg", "dWu", "dWd", "dW_lu", "dWsg", "dWsu",
                  "dWsd", "ws")


class BackwardArgs(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in BWD_ARG_FIELDS] +
                [("ws_bytes", ctypes.c_size_t), ("status", ctypes.c_void_p),
                 ("expert_offsets", ctypes.c_void_p), ("bank", ctypes.c_void_p)])

LAYER_BUFFER_FIELDS = ("Wr", "bias", "W_ld", "Wg", "Wu", "Wd", "W_lu", "Wsg", "Wsu", "Wsd",
                       "logits", "idx", "w", "tie", "z", "ws_dispatch", "ws_dispatch_bytes",
                       "pool", "slot_of", "drop", "expert_rows", "expert_count", "stats", "bank",
                       "ws_ffn", "ws_ffn_bytes", "ypool", "c", "a", "status")


class LayerBuffers(ctypes.Structure):
    _fields_ = [(f, ctypes.c_size_t if f.endswith("_bytes") else ctypes.c_void_p)
                for f in LAYER_BUFFER_FIELDS]


class Norm(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int32), ("res_f32", ctypes.c_int32),
                ("gate_per_token", ctypes.c_int32), ("alpha", ctypes.c_float),
                ("beta", ctypes.c_float), ("eps", ctypes.c_float)]


class RotaryTable(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("rot_dim", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("orig_len", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("magnitude", ctypes.c_double)]


class Rotary(ctypes.Structure):
    _fields_ = ([("T", ctypes.c_int64)] +
                [(f, ctypes.c_int32) for f in ("hq", "hk", "D", "rot_dim", "interleaved",
                                               "inverse")] +
                [(f, ctypes.c_int64) for f in ("table_rows", "q_t", "q_h", "k_t", "k_h", "qo_t",
                                               "qo_h", "ko_t", "ko_h")])


class Attention(ctypes.Structure):
    _fields_ = ([("T", ctypes.c_int64)] +
                [(f, ctypes.c_int32) for f in ("n_seqs", "n_heads", "n_kv_heads", "head_dim")] +
                [("scale", ctypes.c_float), ("reserved", ctypes.c_int32)] +
                [(f, ctypes.c_int64) for f in ("q_t", "q_h", "k_t", "k_h", "v_t", "v_h", "o_t",
                                               "o_h", "do_t", "do_h", "dq_t", "dq_h", "dk_t",
                                               "dk_h", "dv_t", "dv_h")])


class GradTensor(ctypes.Structure):
    _fields_ = [("in", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("is_bf16", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class HeadNorm(ctypes.Structure):
    _fields_ = ([("T", ctypes.c_int64)] +
                [(f, ctypes.c_int32) for f in ("hq", "hk", "D", "rot_dim", "interleaved")] +
                [("eps", ctypes.c_float)] +
                [(f, ctypes.c_int64) for f in ("table_rows", "q_t", "q_h", "k_t", "k_h", "qo_t",
                                               "qo_h", "ko_t", "ko_h", "dq_t", "dq_h", "dk_t",
                                               "dk_h")])


class RoutingConfig(ctypes.Structure):
    _fields_ = ([("T", ctypes.c_int64)] +
                [(f, ctypes.c_int32) for f in ("n_experts", "top_k", "score", "n_groups",
                                               "groups_kept", "group_top", "renorm")] +
                [("scale", ctypes.c_float), ("grad_f32", ctypes.c_int32),
                 ("reserved", ctypes.c_int32)])


class EmbeddingConfig(ctypes.Structure):
    _fields_ = ([("T", ctypes.c_int64), ("V", ctypes.c_int64)] +
                [(f, ctypes.c_int32) for f in ("d", "table_f32", "out_f32", "accumulate")] +
                [("scale", ctypes.c_float), ("reserved", ctypes.c_int32)])


class Distill(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_int64) for f in ("T", "V", "z_ld", "dz_ld")] +
                [(f, ctypes.c_int32) for f in ("K", "z_f32", "teacher_f32")] +
                [("temperature", ctypes.c_float), ("scale", ctypes.c_float),
                 ("reserved", ctypes.c_int32)])


_lib = None


def lib() -> ctypes.CDLL:
    """Load the library once; raise if it has not been built."""
    global _lib
    if _lib is None:
        _lib = load_library(LIB_PATH)
    return _lib


def load_library(path: str) -> ctypes.CDLL:
    """Load one build of the library (e.g. the checked one) with its
    signatures declared; ``lib()`` serves the package's own build."""
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m moe_routing_capacity_gb300.build`")
    L = ctypes.CDLL(path)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    pc = ctypes.POINTER(Config)
    L.moe_plan.argtypes = [pc, ctypes.POINTER(Plan)]
    L.moe_router_topk.argtypes = [pc, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_latent_proj.argtypes = [vp, vp, i64, i32, i32, vp, vp, vp]
    L.moe_route_project.argtypes = [pc, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_matmul.argtypes = [vp, ctypes.c_int, i64, vp, ctypes.c_int, i64, i64, i32, i32, vp,
                             ctypes.c_int, i64, vp, vp]
    L.moe_dispatch_pooled.argtypes = [pc, vp, vp, vp, sz, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_dispatch_pooled_noalloc.argtypes = [pc, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_expert_ffn_grouped.argtypes = [pc, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp]
    L.moe_combine.argtypes = [pc, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_dispatch_expert_waves.argtypes = [pc, vp, vp, vp, sz, vp, vp, vp, vp, vp, vp, vp, vp,
                                            vp, vp, sz, vp, vp, vp]
    L.moe_dispatch_shared_overlap.argtypes = [pc, vp, vp, vp, sz, vp, vp, vp, vp, vp, vp, vp, vp,
                                              vp, vp, vp, vp, vp]
    L.moe_balance_update.argtypes = [pc, vp, vp, ctypes.c_float, vp, vp]
    L.moe_balance_update_window.argtypes = [pc, vp, vp, vp, i32, vp, ctypes.c_float, vp, vp]
    L.moe_plan_ragged.argtypes = [pc, ctypes.POINTER(Plan)]
    L.moe_dispatch_ragged.argtypes = [pc, vp, vp, vp, sz, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_dispatch_ragged_shared_overlap.argtypes = [pc, vp, vp, vp, sz, vp, vp, vp, vp, vp, vp,
                                                     vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_expert_ffn_ragged.argtypes = [pc, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp]
    L.moe_backward_plan.argtypes = [pc, ctypes.POINTER(BackwardWs)]
    L.moe_layer_backward.argtypes = [pc, ctypes.POINTER(BackwardArgs), vp]
    L.moe_backward_plan_ragged.argtypes = [pc, ctypes.POINTER(BackwardWs)]
    L.moe_layer_backward_ragged.argtypes = [pc, ctypes.POINTER(BackwardArgs), vp]
    L.moe_strerror.argtypes = [ctypes.c_int]
    L.moe_strerror.restype = ctypes.c_char_p
    L.moe_abi_version.argtypes = []
    L.moe_check_status.argtypes = []
    L.moe_trace_begin.argtypes = [ctypes.c_int]
    L.moe_trace_mark.argtypes = [vp]
    L.moe_trace_end.argtypes = []
    L.moe_trace_event.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_char_p),
                                  ctypes.POINTER(ctypes.c_float)]
    for n in EXPORTS:
        if n != "moe_strerror":
            getattr(L, n).restype = ctypes.c_int
    pb = ctypes.POINTER(LayerBuffers)
    L.moe_layer_forward.argtypes = [pc, pb, vp, vp, vp]
    L.moe_host_pipe_create.argtypes = [pc, ctypes.c_int, ctypes.POINTER(vp), ctypes.POINTER(vp),
                                       ctypes.POINTER(vp), ctypes.POINTER(vp)]
    L.moe_host_pipe_submit.argtypes = [vp, pb, vp, vp, vp, vp]
    L.moe_host_pipe_sync.argtypes = [vp]
    L.moe_host_pipe_destroy.argtypes = [vp]
    pi64 = ctypes.POINTER(i64)
    pn, pa = ctypes.POINTER(Norm), ctypes.POINTER(Attention)
    L.moe_norm_residual.argtypes = [pn] + [vp] * 10
    L.moe_norm_residual_workspace.argtypes = [i64, i32, pi64]
    L.moe_norm_residual_backward.argtypes = [pn] + [vp] * 15 + [i64, vp]
    L.moe_rotary_make_table.argtypes = [ctypes.POINTER(RotaryTable), vp, vp]
    L.moe_rotary.argtypes = [ctypes.POINTER(Rotary)] + [vp] * 8
    L.moe_attention_workspace.argtypes = [pa, pi64, pi64]
    L.moe_attention_plan.argtypes = [pa, vp, vp, i64, vp, vp]
    L.moe_attention_forward.argtypes = [pa] + [vp] * 9
    L.moe_attention_backward.argtypes = [pa] + [vp] * 12 + [i64, vp, vp]
    L.moe_grad_clip_workspace.argtypes = [i64, pi64]
    L.moe_grad_clip.argtypes = [ctypes.POINTER(GradTensor), i64, ctypes.c_float, vp, vp, i64, vp]
    ph, pr = ctypes.POINTER(HeadNorm), ctypes.POINTER(RoutingConfig)
    pe, pd = ctypes.POINTER(EmbeddingConfig), ctypes.POINTER(Distill)
    L.moe_head_norm_rotary.argtypes = [ph] + [vp] * 10
    L.moe_head_norm_rotary_workspace.argtypes = [i64, i32, i32, i32, pi64]
    L.moe_head_norm_rotary_backward.argtypes = [ph] + [vp] * 13 + [i64, vp, vp]
    L.moe_route_logits.argtypes = [pc] + [vp] * 7
    L.moe_layer_backward_routed.argtypes = [pc, ctypes.c_int, ctypes.POINTER(BackwardArgs), pr,
                                            vp, vp]
    L.moe_router_select.argtypes = [pr] + [vp] * 5
    L.moe_router_select_backward.argtypes = [pr] + [vp] * 5
    L.moe_embedding.argtypes = [pe] + [vp] * 5
    L.moe_embedding_workspace.argtypes = [i64, i64, i32, pi64]
    L.moe_embedding_plan.argtypes = [i64, i64, i32, vp, vp, i64, vp, vp]
    L.moe_embedding_backward.argtypes = [pe, vp, i64, vp, vp, vp]
    L.moe_distill_loss.argtypes = [pd] + [vp] * 10
    L.moe_distill_loss_backward.argtypes = [pd] + [vp] * 8
    if hasattr(L, "moe_check_set_wave_wait_limit_ns"):
        L.moe_check_set_wave_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
        L.moe_check_set_wave_wait_limit_ns.restype = ctypes.c_int
    return L


def strerror(code: int) -> str:
    return lib().moe_strerror(code).decode()


def make_config(cfg) -> Config:
    """C config from any object with the layer-size attributes."""
    return Config(cfg.T, cfg.d_model, cfg.d_latent, cfg.n_experts, cfg.n_ranks, cfg.top_k,
                  cfg.n_waves, cfg.n_shared, cfg.h_expert, cfg.h_shared, 0,
                  float(cfg.cf_send), float(cfg.cf_recv))


def plan(cfg) -> Plan:
    p = Plan()
    rc = lib().moe_plan(ctypes.byref(make_config(cfg)), ctypes.byref(p))
    if rc:
        raise MoeError("moe_plan", rc)
    return p


def plan_ragged(cfg) -> Plan:
    p = Plan()
    rc = lib().moe_plan_ragged(ctypes.byref(make_config(cfg)), ctypes.byref(p))
    if rc:
        raise MoeError("moe_plan_ragged", rc)
    return p


def _ptr(t, dtype=None, allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise ValueError("tensor required")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:   # the current stream's handle, without building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def on_stream(stream=None):
    """Context in which tensors are allocated and cleared for use on ``stream``
    (None: the current one).  Memory taken under another stream's name may
    still be written by work queued there."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _check(fn, rc):
    if rc:
        raise MoeError(fn, rc)


bf16, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def router_topk(cfg, x, Wr, bias, logits, idx, w, tie, status, stream=None):
    _check("moe_router_topk", lib().moe_router_topk(
        ctypes.byref(make_config(cfg)), _ptr(x, bf16), _ptr(Wr, bf16),
        _ptr(bias, f32, allow_none=True), _ptr(logits, f32), _ptr(idx, i32), _ptr(w, f32),
        _ptr(tie, u8), _ptr(status, i32), _stream(stream)))


def latent_proj(inp, W, out, status, stream=None):
    M, K = inp.shape
    N = W.shape[0]
    if W.shape[1] != K or tuple(out.shape) != (M, N):
        raise ValueError("shape mismatch")
    _check("moe_latent_proj", lib().moe_latent_proj(
        _ptr(inp, bf16), _ptr(W, bf16), M, K, N, _ptr(out, bf16), _ptr(status, i32),
        _stream(stream)))


def matmul(A, B, M, N, K, out, status, a_mn=False, b_mn=False, stream=None):
    """out[M, N] = sum_k A(m, k) B(n, k); A stored [M, K] (or [K, M] if a_mn),
    B stored [N, K] (or [K, N] if b_mn); out bf16 or fp32, row-major."""
    lda, ldb = A.shape[1], B.shape[1]
    _check("moe_matmul", lib().moe_matmul(
        _ptr(A, bf16), int(bool(a_mn)), lda, _ptr(B, bf16), int(bool(b_mn)), ldb, M, N, K,
        _ptr(out), int(out.dtype == torch.float32), out.shape[1], _ptr(status, i32),
        _stream(stream)))


def route_project(cfg, x, Wr, bias, W_ld, logits, idx, w, tie, z, status, stream=None):
    _check("moe_route_project", lib().moe_route_project(
        ctypes.byref(make_config(cfg)), _ptr(x, bf16), _ptr(Wr, bf16),
        _ptr(bias, f32, allow_none=True), _ptr(W_ld, bf16), _ptr(logits, f32), _ptr(idx, i32),
        _ptr(w, f32), _ptr(tie, u8), _ptr(z, bf16), _ptr(status, i32), _stream(stream)))


def route_logits(cfg, x, Wr, W_ld, logits, z, status, stream=None):
    """logits = x Wr^T and the latent projection z in one pass over x, for
    router_select's choice (W_ld, z None: the logits alone)."""
    _check("moe_route_logits", lib().moe_route_logits(
        ctypes.byref(make_config(cfg)), _ptr(x, bf16), _ptr(Wr, bf16),
        _ptr(W_ld, bf16, allow_none=True), _ptr(logits, f32), _ptr(z, bf16, allow_none=True),
        _ptr(status, i32), _stream(stream)))


def dispatch_pooled(cfg, z, idx, ws, pool, slot_of, drop, expert_rows, expert_count, stats,
                    stream=None, bank=None):
    """bank (optional, [E, c_recv, L] bf16): also receives each receiver-kept
    row at its expert's receiver rank."""
    _check("moe_dispatch_pooled", lib().moe_dispatch_pooled(
        ctypes.byref(make_config(cfg)), _ptr(z, bf16), _ptr(idx, i32), _ptr(ws, u8),
        ws.numel(), _ptr(pool, torch.int16), _ptr(slot_of, i32), _ptr(drop, u8),
        _ptr(expert_rows, i32), _ptr(expert_count, i32), _ptr(stats, torch.int64),
        _ptr(bank, bf16, allow_none=True), _stream(stream)))


# MOE_DISPATCH_NOALLOC_SCRATCH_BYTES of the header (a host test checks that
# the two agree)
NOALLOC_SCRATCH_BYTES = 8 << 20


def dispatch_pooled_noalloc(cfg, z, idx, pool, slot_of, drop, expert_rows, expert_count, stats,
                            stream=None):
    """moe_dispatch_pooled with the library's fixed scratch array instead of a
    caller-provided one (for callers that cannot allocate device memory)."""
    _check("moe_dispatch_pooled_noalloc", lib().moe_dispatch_pooled_noalloc(
        ctypes.byref(make_config(cfg)), _ptr(z, bf16), _ptr(idx, i32),
        _ptr(pool, torch.int16), _ptr(slot_of, i32), _ptr(drop, u8), _ptr(expert_rows, i32),
        _ptr(expert_count, i32), _ptr(stats, torch.int64), _stream(stream)))


def expert_ffn_grouped(cfg, pool, expert_rows, expert_count, Wg, Wu, Wd, ws, ypool, status,
                       stream=None, bank=None):
    """bank (optional): the per-expert rows the dispatch wrote; None gathers
    the rows from the pool."""
    _check("moe_expert_ffn_grouped", lib().moe_expert_ffn_grouped(
        ctypes.byref(make_config(cfg)), _ptr(pool, torch.int16),
        _ptr(bank, bf16, allow_none=True), _ptr(expert_rows, i32),
        _ptr(expert_count, i32), _ptr(Wg, bf16), _ptr(Wu, bf16), _ptr(Wd, bf16),
        _ptr(ws, u8), ws.numel(), _ptr(ypool, bf16), _ptr(status, i32), _stream(stream)))


def dispatch_expert_waves(cfg, z, idx, ws, pool, slot_of, drop, expert_rows, expert_count, stats,
                          Wg, Wu, Wd, ffn_ws, ypool, status, stream=None):
    """dispatch_pooled then expert_ffn_grouped, with the later waves' pool rows
    copied inside the gate/up launch while wave 0's experts compute."""
    _check("moe_dispatch_expert_waves", lib().moe_dispatch_expert_waves(
        ctypes.byref(make_config(cfg)), _ptr(z, bf16), _ptr(idx, i32), _ptr(ws, u8),
        ws.numel(), _ptr(pool, torch.int16), _ptr(slot_of, i32), _ptr(drop, u8),
        _ptr(expert_rows, i32), _ptr(expert_count, i32), _ptr(stats, torch.int64),
        _ptr(Wg, bf16), _ptr(Wu, bf16), _ptr(Wd, bf16), _ptr(ffn_ws, u8), ffn_ws.numel(),
        _ptr(ypool, bf16), _ptr(status, i32), _stream(stream)))


def dispatch_shared_overlap(cfg, z, idx, ws, pool, slot_of, drop, expert_rows, expert_count,
                            stats, x, Wsg, Wsu, a, status, stream=None, bank=None):
    """dispatch_pooled plus the shared experts' activations a, the pool rows
    copied while the shared gate/up product computes; then call combine with
    Wsg = Wsu = None."""
    _check("moe_dispatch_shared_overlap", lib().moe_dispatch_shared_overlap(
        ctypes.byref(make_config(cfg)), _ptr(z, bf16), _ptr(idx, i32), _ptr(ws, u8),
        ws.numel(), _ptr(pool, torch.int16), _ptr(slot_of, i32), _ptr(drop, u8),
        _ptr(expert_rows, i32), _ptr(expert_count, i32), _ptr(stats, torch.int64),
        _ptr(bank, bf16, allow_none=True),
        _ptr(x, bf16, allow_none=True), _ptr(Wsg, bf16, allow_none=True),
        _ptr(Wsu, bf16, allow_none=True), _ptr(a, bf16, allow_none=True), _ptr(status, i32),
        _stream(stream)))


def dispatch_ragged(cfg, z, idx, ws, pool, slot_of, drop, expert_offsets, expert_rows,
                    expert_count, stats, stream=None, bank=None):
    _check("moe_dispatch_ragged", lib().moe_dispatch_ragged(
        ctypes.byref(make_config(cfg)), _ptr(z, bf16), _ptr(idx, i32), _ptr(ws, u8),
        ws.numel(), _ptr(pool, torch.int16), _ptr(slot_of, i32), _ptr(drop, u8),
        _ptr(expert_offsets, i32), _ptr(expert_rows, i32), _ptr(expert_count, i32),
        _ptr(stats, torch.int64), _ptr(bank, bf16, allow_none=True), _stream(stream)))


def dispatch_ragged_shared_overlap(cfg, z, idx, ws, pool, slot_of, drop, expert_offsets,
                                   expert_rows, expert_count, stats, x, Wsg, Wsu, a, status,
                                   stream=None, bank=None):
    """dispatch_ragged plus the shared experts' activations a, the pack run
    inside the shared gate/up product; then call combine with Wsg = Wsu = None."""
    _check("moe_dispatch_ragged_shared_overlap", lib().moe_dispatch_ragged_shared_overlap(
        ctypes.byref(make_config(cfg)), _ptr(z, bf16), _ptr(idx, i32), _ptr(ws, u8),
        ws.numel(), _ptr(pool, torch.int16), _ptr(slot_of, i32), _ptr(drop, u8),
        _ptr(expert_offsets, i32), _ptr(expert_rows, i32), _ptr(expert_count, i32),
        _ptr(stats, torch.int64), _ptr(bank, bf16, allow_none=True),
        _ptr(x, bf16, allow_none=True), _ptr(Wsg, bf16, allow_none=True),
        _ptr(Wsu, bf16, allow_none=True), _ptr(a, bf16, allow_none=True), _ptr(status, i32),
        _stream(stream)))


def expert_ffn_ragged(cfg, pool, expert_offsets, expert_rows, expert_count, Wg, Wu, Wd, ws,
                      ypool, status, stream=None, bank=None):
    _check("moe_expert_ffn_ragged", lib().moe_expert_ffn_ragged(
        ctypes.byref(make_config(cfg)), _ptr(pool, torch.int16),
        _ptr(bank, bf16, allow_none=True), _ptr(expert_offsets, i32),
        _ptr(expert_rows, i32), _ptr(expert_count, i32), _ptr(Wg, bf16), _ptr(Wu, bf16),
        _ptr(Wd, bf16), _ptr(ws, u8), ws.numel(), _ptr(ypool, bf16), _ptr(status, i32),
        _stream(stream)))


def balance_update(cfg, idx, hist, alpha, bias, stream=None):
    _check("moe_balance_update", lib().moe_balance_update(
        ctypes.byref(make_config(cfg)), _ptr(idx, i32), _ptr(hist, torch.int64),
        float(alpha), _ptr(bias, f32), _stream(stream)))


def balance_update_window(cfg, idx, hist, ring, step, alpha, bias, stream=None):
    """moe_balance_update over exactly the past ring.shape[0] batches (ring
    [N, E] int64 and step [1] int64 live on the device, zero at the start)."""
    _check("moe_balance_update_window", lib().moe_balance_update_window(
        ctypes.byref(make_config(cfg)), _ptr(idx, i32), _ptr(hist, torch.int64),
        _ptr(ring, torch.int64), int(ring.shape[0]), _ptr(step, torch.int64), float(alpha),
        _ptr(bias, f32), _stream(stream)))


def combine(cfg, ypool, slot_of, w, W_lu, x, Wsg, Wsu, Wsd, c, a, out, status, stream=None):
    _check("moe_combine", lib().moe_combine(
        ctypes.byref(make_config(cfg)), _ptr(ypool, bf16), _ptr(slot_of, i32), _ptr(w, f32),
        _ptr(W_lu, bf16), _ptr(x, bf16, allow_none=True), _ptr(Wsg, bf16, allow_none=True),
        _ptr(Wsu, bf16, allow_none=True), _ptr(Wsd, bf16, allow_none=True),
        _ptr(c, bf16), _ptr(a, bf16, allow_none=True), _ptr(out, bf16), _ptr(status, i32),
        _stream(stream)))


def stats_dict(stats_tensor) -> dict:
    """Decode a moe_drop_stats_t record held in an int64 tensor of STATS_WORDS."""
    raw = bytes(stats_tensor.detach().cpu().numpy().tobytes())
    s = DropStats.from_buffer_copy(raw)
    return {f: getattr(s, f) for f, _ in DropStats._fields_}


# ---------------------------------------------------------------- whole layer

def layer_buffers(tensors: dict) -> LayerBuffers:
    """moe_layer_buffers_t from tensors named as its fields (None: NULL); the
    two sizes are taken from the scratch tensors."""
    b = LayerBuffers()
    for f in LAYER_BUFFER_FIELDS:
        if f.endswith("_bytes"):
            t = tensors.get(f[: -len("_bytes")])
            setattr(b, f, t.numel() * t.element_size() if t is not None else 0)
            continue
        t = tensors.get(f)
        if t is not None:
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{f}: contiguous device tensor required")
            setattr(b, f, t.data_ptr())
    return b


def layer_forward(cfg, buffers: LayerBuffers, x, out, stream=None):
    _check("moe_layer_forward", lib().moe_layer_forward(
        ctypes.byref(make_config(cfg)), ctypes.byref(buffers), _ptr(x, bf16), _ptr(out, bf16),
        _stream(stream)))


class HostPipe:
    """moe_host_pipe_*: batches from host memory through moe_layer_forward,
    the copies on the pipeline's own streams.  x_dev, out_dev, stats_dev:
    lists of device staging tensors (the ring)."""

    def __init__(self, cfg, x_dev, out_dev, stats_dev):
        self.cfg = make_config(cfg)
        n = len(x_dev)
        arr = lambda ts: (ctypes.c_void_p * n)(*[t.data_ptr() for t in ts])
        self._keep = (x_dev, out_dev, stats_dev)
        self.h = ctypes.c_void_p()
        _check("moe_host_pipe_create", lib().moe_host_pipe_create(
            ctypes.byref(self.cfg), n, arr(x_dev), arr(out_dev), arr(stats_dev),
            ctypes.byref(self.h)))

    def submit(self, buffers: LayerBuffers, x_host, out_host, stats_host=None, stream=None):
        for t in (x_host, out_host) + ((stats_host,) if stats_host is not None else ()):
            if t.is_cuda or not t.is_contiguous():
                raise ValueError("host tensors required (pinned for overlap)")
        _check("moe_host_pipe_submit", lib().moe_host_pipe_submit(
            self.h, ctypes.byref(buffers), ctypes.c_void_p(x_host.data_ptr()),
            ctypes.c_void_p(out_host.data_ptr()),
            ctypes.c_void_p(stats_host.data_ptr()) if stats_host is not None else None,
            _stream(stream)))

    def synchronize(self):
        _check("moe_host_pipe_sync", lib().moe_host_pipe_sync(self.h))

    def close(self):
        if self.h:
            rc = lib().moe_host_pipe_destroy(self.h)
            self.h = ctypes.c_void_p()
            _check("moe_host_pipe_destroy", rc)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------- timing trace

def trace_begin(n: int):
    _check("moe_trace_begin", lib().moe_trace_begin(n))


def trace_mark(stream=None):
    _check("moe_trace_mark", lib().moe_trace_mark(_stream(stream)))


def trace_end() -> list:
    """Stop tracing; return [(kernel name, ms since the previous event)]."""
    n = lib().moe_trace_end()
    out = []
    name = ctypes.c_char_p()
    ms = ctypes.c_float()
    for i in range(n):
        _check("moe_trace_event", lib().moe_trace_event(i, ctypes.byref(name), ctypes.byref(ms)))
        out.append((name.value.decode(), float(ms.value)))
    return out


# ---------------------------------------------------------------- backward pass

def backward_plan(cfg, ragged=False) -> BackwardWs:
    w = BackwardWs()
    fn = "moe_backward_plan_ragged" if ragged else "moe_backward_plan"
    _check(fn, getattr(lib(), fn)(ctypes.byref(make_config(cfg)), ctypes.byref(w)))
    return w


def layer_backward(cfg, tensors: dict, ws, status, stream=None, routing=None, logits=None):
    """tensors: every BackwardArgs field by name (torch tensors, or None for
    the shared-expert ones when there are none).  routing, logits: the rule and
    the input of router_select, where the experts were chosen by it."""
    args = BackwardArgs()
    for f in BWD_ARG_FIELDS:
        t = tensors.get(f)
        setattr(args, f, None if t is None else t.data_ptr())
    args.ws = ws.data_ptr()
    args.ws_bytes = ws.numel()
    args.status = status.data_ptr()
    eoff = tensors.get("expert_offsets")
    args.expert_offsets = None if eoff is None else eoff.data_ptr()
    bank = tensors.get("bank")
    args.bank = None if bank is None else bank.data_ptr()
    if routing is not None:
        _check("moe_layer_backward_routed", lib().moe_layer_backward_routed(
            ctypes.byref(make_config(cfg)), int(eoff is not None), ctypes.byref(args),
            ctypes.byref(routing.config(cfg.T)), _ptr(logits, f32), _stream(stream)))
        return
    fn = "moe_layer_backward" if eoff is None else "moe_layer_backward_ragged"
    _check(fn, getattr(lib(), fn)(ctypes.byref(make_config(cfg)), ctypes.byref(args),
                                  _stream(stream)))


# ---------------------------------------------------------------- training block

def _rows(name, t, shape, dtypes, allow_none=False):
    """Device address of a contiguous tensor of this shape and one of these types."""
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name}: tensor required")
    # one condition where all is well: a small call's time is mostly these
    if t.dtype in dtypes and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name}: contiguous device tensor required")


_BF16, _F32, _RES, _I32 = (bf16,), (f32,), (bf16, f32), (i32,)


def _norm_config(r, gate, alpha, beta, eps):
    rows = r.shape
    if len(rows) != 2:
        raise ValueError("the residual stream is [T, d]")
    T, d = rows
    per_token = gate is not None and gate.dim() == 2
    return rows, (d,), (T,), Norm(T, d, r.dtype == f32, per_token, alpha, beta, eps)


def norm_residual(b, r, gate, w_post, w_pre, y, n, rstd_post=None, rstd_pre=None, alpha=1.0,
                  beta=1.0, eps=1e-6, stream=None):
    """y = alpha r + beta gate (norm(b) w_post), n = norm(y) w_pre, in one pass:
    the norm after a branch (output b [T, d] bf16, or None: y = alpha r), its
    gate ([d], [T, d] or None), the residual sum (r, y [T, d] bf16 or fp32; y
    may be r, or None) and the norm before the next branch (n [T, d] bf16, or
    None).  rstd_post, rstd_pre [T] fp32 receive the statistics that the
    backward reads (None: not wanted)."""
    rows, chan, tok, c = _norm_config(r, gate, alpha, beta, eps)
    _check("moe_norm_residual", lib().moe_norm_residual(
        ctypes.byref(c), _rows("b", b, rows, _BF16, True), _rows("r", r, rows, _RES),
        _rows("gate", gate, rows if c.gate_per_token else chan, _BF16, True),
        _rows("w_post", w_post, chan, _BF16, True), _rows("w_pre", w_pre, chan, _BF16, True),
        _rows("y", y, rows, (r.dtype,), True), _rows("n", n, rows, _BF16, True),
        _rows("rstd_post", rstd_post, tok, _F32, True),
        _rows("rstd_pre", rstd_pre, tok, _F32, True), _stream(stream)))


def norm_residual_workspace(T, d) -> int:
    """Scratch bytes of norm_residual_backward."""
    v = ctypes.c_int64()
    _check("moe_norm_residual_workspace",
           lib().moe_norm_residual_workspace(T, d, ctypes.byref(v)))
    return v.value


def norm_residual_backward(dn, dy, b, r, gate, w_post, w_pre, rstd_post, rstd_pre, db, dr, dgate,
                           dw_post, dw_pre, ws, alpha=1.0, beta=1.0, stream=None):
    """Gradients of norm_residual for dn (of n) and dy (of y, the part that
    passes this norm by; None: zero): db, dr (may be dy), dgate ([d] fp32 for
    a [d] gate, else [T, d] bf16), dw_post, dw_pre [d] fp32.  None exactly
    where the forward's tensor is."""
    rows, chan, tok, c = _norm_config(dr, gate, alpha, beta, 0.0)
    rt, at = (dr.dtype,), rows if c.gate_per_token else chan
    _check("moe_norm_residual_backward", lib().moe_norm_residual_backward(
        ctypes.byref(c), _rows("dn", dn, rows, _BF16, True), _rows("dy", dy, rows, rt, True),
        _rows("b", b, rows, _BF16, True), _rows("r", r, rows, rt, True),
        _rows("gate", gate, at, _BF16, True), _rows("w_post", w_post, chan, _BF16, True),
        _rows("w_pre", w_pre, chan, _BF16, True), _rows("rstd_post", rstd_post, tok, _F32, True),
        _rows("rstd_pre", rstd_pre, tok, _F32, True), _rows("db", db, rows, _BF16, True),
        _rows("dr", dr, rows, _RES),
        _rows("dgate", dgate, at, _BF16 if c.gate_per_token else _F32, True),
        _rows("dw_post", dw_post, chan, _F32, True), _rows("dw_pre", dw_pre, chan, _F32, True),
        _ptr(ws, u8), ws.numel(), _stream(stream)))


ROTARY_SCALING = {"none": 0, "linear": 1, "base": 2, "by_parts": 3}


def rotary_table(table, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, beta_fast=32.0,
                 beta_slow=1.0, magnitude=1.0, stream=None):
    """Fill table [positions, rot_dim / 2, 2] fp32 with {cos, sin} of the
    rotary angles (see moe_rotary_make_table for the scalings)."""
    if table.dim() != 3 or table.shape[2] != 2:
        raise ValueError("the table is [positions, rot_dim / 2, 2]")
    if scaling not in ROTARY_SCALING:
        raise ValueError(f"scaling must be one of {sorted(ROTARY_SCALING)}")
    c = RotaryTable(table.shape[0], 2 * table.shape[1], ROTARY_SCALING[scaling], base, factor,
                    orig_len, beta_fast, beta_slow, magnitude)
    _check("moe_rotary_make_table", lib().moe_rotary_make_table(
        ctypes.byref(c), _ptr(table, f32), _stream(stream)))


def _heads(name, t, shape):
    """(address, token stride, head stride) of a [T, heads, D] bf16 tensor
    whose channels are contiguous (tokens and heads may be strided)."""
    if t.dtype == bf16 and t.shape == shape:
        st, sh, sd = t.stride()
        if sd == 1 and t.is_cuda:
            return t.data_ptr(), st, sh
        raise ValueError(f"{name}: device tensor with contiguous channels required")
    if t.dtype != bf16:
        raise TypeError(f"{name}: expected {bf16}, got {t.dtype}")
    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")


def rotary(q, k, table, pos, q_out, k_out, status, interleaved=False, inverse=False, stream=None):
    """Turn the first 2 table.shape[1] channels of every head of q [T, hq, D]
    and k [T, hk, D] (None: no keys) to the tokens' positions pos [T] int32
    (None: 0, 1, ...), into q_out and k_out (which may be q and k).  inverse:
    the gradient's direction.  interleaved: pairs side by side."""
    T, hq, D = q.shape
    hk = 0 if k is None else k.shape[1]
    qs, ks = (T, hq, D), (T, hk, D)
    qp, qt, qh = _heads("q", q, qs)
    qop, qot, qoh = _heads("q_out", q_out, qs)
    kp, kt, kh = (None, 0, 0) if k is None else _heads("k", k, ks)
    kop, kot, koh = (None, 0, 0) if k is None else _heads("k_out", k_out, ks)
    if table.dim() != 3 or table.shape[2] != 2:
        raise ValueError("the table is [positions, rot_dim / 2, 2]")
    if pos is not None and tuple(pos.shape) != (T,):
        raise ValueError("pos is [T]")
    c = Rotary(T, hq, hk, D, 2 * table.shape[1], int(bool(interleaved)), int(bool(inverse)),
               table.shape[0], qt, qh, kt, kh, qot, qoh, kot, koh)
    _check("moe_rotary", lib().moe_rotary(
        ctypes.byref(c), qp, kp, _ptr(table, f32), _ptr(pos, i32, allow_none=True), qop, kop,
        _ptr(status, i32), _stream(stream)))


class AttentionPlan:
    """Work lists of one batch of packed sequences: sequence s is the tokens
    cu_seqlens[s] .. cu_seqlens[s + 1) of T (int32 on the device, read on the
    stream, never on the host).  It serves any number of attention and
    attention_backward calls of these sizes; refill() takes another batch's
    cu_seqlens of the same length.  ``status`` receives MOE_EINVAL if they
    decrease or leave [0, T]; calls on such a plan write nothing and set their
    own status likewise."""

    def __init__(self, cu_seqlens, T, n_heads, n_kv_heads, head_dim, status=None, stream=None):
        self.T, self.n_heads, self.n_kv_heads, self.head_dim = T, n_heads, n_kv_heads, head_dim
        self.n_seqs = cu_seqlens.numel() - 1
        if cu_seqlens.dim() != 1 or self.n_seqs < 0:
            raise ValueError("cu_seqlens is [sequences + 1]")
        pb, bb = ctypes.c_int64(), ctypes.c_int64()
        _check("moe_attention_workspace", lib().moe_attention_workspace(
            ctypes.byref(self._config()), ctypes.byref(pb), ctypes.byref(bb)))
        self.backward_ws_bytes = bb.value
        with on_stream(stream):
            self.status = (torch.zeros(1, dtype=i32, device=cu_seqlens.device) if status is None
                           else status)
            self.plan = torch.empty(pb.value, dtype=u8, device=cu_seqlens.device)
        self.address = self.plan.data_ptr()
        self.q_shape, self.k_shape = (T, n_heads, head_dim), (T, n_kv_heads, head_dim)
        self.lse_shape = (n_heads, T)
        self.refill(cu_seqlens, stream)

    def _config(self, scale=None):
        return Attention(self.T, self.n_seqs, self.n_heads, self.n_kv_heads, self.head_dim,
                         self.head_dim ** -0.5 if scale is None else scale)

    def refill(self, cu_seqlens, stream=None):
        if tuple(cu_seqlens.shape) != (self.n_seqs + 1,):
            raise ValueError("cu_seqlens of another number of sequences")
        _check("moe_attention_plan", lib().moe_attention_plan(
            ctypes.byref(self._config()), _ptr(cu_seqlens, i32), _ptr(self.plan, u8),
            self.plan.numel(), _ptr(self.status, i32), _stream(stream)))


def attention(plan, q, k, v, out, lse, status, scale=None, rest=None, stream=None):
    """Causal attention within each of the plan's sequences: q, out [T,
    n_heads, D], k, v [T, n_kv_heads, D] bf16 (strided views allowed), lse
    [n_heads, T] fp32; scale D^-1/2 unless given.  rest (like out): what
    rounding took from out, for attention_backward (None: no gradient)."""
    c = plan._config(scale)
    qs, ks = plan.q_shape, plan.k_shape
    qp, c.q_t, c.q_h = _heads("q", q, qs)
    kp, c.k_t, c.k_h = _heads("k", k, ks)
    vp, c.v_t, c.v_h = _heads("v", v, ks)
    op, c.o_t, c.o_h = _heads("out", out, qs)
    rp = None if rest is None else _rest(rest, qs, c)
    _check("moe_attention_forward", lib().moe_attention_forward(
        ctypes.byref(c), plan.address, qp, kp, vp, op, rp, _rows("lse", lse, plan.lse_shape, _F32),
        _ptr(status, i32), _stream(stream)))


def _rest(rest, shape, c):
    p, st, sh = _heads("rest", rest, shape)
    if (st, sh) != (c.o_t, c.o_h):
        raise ValueError("rest has out's strides")
    return p


def attention_backward(plan, q, k, v, out, rest, lse, dout, dq, dk, dv, ws, status, scale=None,
                       stream=None):
    """dq, dk, dv of attention for the upstream gradient dout, from the
    forward's inputs and its out, rest and lse; ws: plan.backward_ws_bytes."""
    c = plan._config(scale)
    qs, ks = plan.q_shape, plan.k_shape
    qp, c.q_t, c.q_h = _heads("q", q, qs)
    kp, c.k_t, c.k_h = _heads("k", k, ks)
    vp, c.v_t, c.v_h = _heads("v", v, ks)
    op, c.o_t, c.o_h = _heads("out", out, qs)
    dop, c.do_t, c.do_h = _heads("dout", dout, qs)
    dqp, c.dq_t, c.dq_h = _heads("dq", dq, qs)
    dkp, c.dk_t, c.dk_h = _heads("dk", dk, ks)
    dvp, c.dv_t, c.dv_h = _heads("dv", dv, ks)
    _check("moe_attention_backward", lib().moe_attention_backward(
        ctypes.byref(c), plan.address, qp, kp, vp, op, _rest(rest, qs, c),
        _rows("lse", lse, plan.lse_shape, _F32), dop, dqp, dkp, dvp, _ptr(ws, u8), ws.numel(),
        _ptr(status, i32), _stream(stream)))


class GradSet:
    """The gradients of one model: contiguous fp32 or bf16 tensors, and where
    the clipped ones go (``outs``; None: in place).  Holds the tensors, and
    scratch for calls on ``stream``."""

    def __init__(self, tensors, outs=None, stream=None):
        outs = tensors if outs is None else outs
        if len(tensors) != len(outs):
            raise ValueError("one output a tensor")
        self.tensors, self.outs = list(tensors), list(outs)
        self.records = (GradTensor * max(1, len(self.tensors)))()
        for r, a, b in zip(self.records, self.tensors, self.outs):
            if a.dtype not in (bf16, f32) or b.dtype != a.dtype or b.shape != a.shape:
                raise TypeError("fp32 or bf16 gradients, each with an output of its own type "
                                "and shape")
            setattr(r, "in", _ptr(a))
            r.out = _ptr(b)
            r.numel, r.is_bf16 = a.numel(), int(a.dtype == bf16)
        v = ctypes.c_int64()
        _check("moe_grad_clip_workspace",
               lib().moe_grad_clip_workspace(len(self.tensors), ctypes.byref(v)))
        dev = self.tensors[0].device if self.tensors else None
        with on_stream(stream):
            self.ws = torch.empty(max(1, v.value), dtype=u8, device=dev) if dev else None


def grad_clip(grads, max_norm, norm, stream=None):
    """norm[0] = the 2-norm over all tensors of the GradSet; each is scaled by
    min(1, max_norm / (norm + 1e-6)) into its output.  A norm that is not
    finite leaves the gradients as they are."""
    ws = grads.ws
    _check("moe_grad_clip", lib().moe_grad_clip(
        grads.records, len(grads.tensors), max_norm, _ptr(norm, f32),
        _ptr(ws, u8, allow_none=True), 0 if ws is None else ws.numel(), _stream(stream)))


# ---------------------------------------------------------------- head norms with rotation

def _at(t, dtype):
    """_ptr's checks; the plain address (None stays None)."""
    if t is not None and t.dtype == dtype and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    return _ptr(t, dtype, allow_none=True)


def _head_norm_shapes(q, k, table, pos):
    """The shapes of q, k and the weights; what HeadNorm needs of the rotation."""
    qs, ks = q.shape, None if k is None else k.shape
    if len(qs) != 3 or (ks is not None and len(ks) != 3):
        raise ValueError("q and k are [T, heads, D]")
    T, _, D = qs
    rot = rows = 0
    if table is not None:
        angles = table.shape
        if len(angles) != 3 or angles[2] != 2:
            raise ValueError("the table is [positions, rot_dim / 2, 2]")
        rows, rot = angles[0], 2 * angles[1]
    if pos is not None and pos.shape != (T,):
        raise ValueError("pos is [T]")
    return qs, ks and (T, ks[1], D), (D,), rot, rows


def head_norm_rotary(q, k, w_q, w_k, table, pos, q_out, k_out, status, eps=1e-6,
                     interleaved=False, stream=None):
    """The norm of every head of q [T, hq, D] (weight w_q [D]) and k [T, hk, D]
    (w_k; None both: no keys), and its rotation as rotary's to the tokens'
    positions pos [T] int32 (None: 0, 1, ...), in one pass into q_out and k_out
    (which may be q and k).  table None: the norm alone."""
    qs, ks, chan, rot, rows = _head_norm_shapes(q, k, table, pos)
    T, hq, D = qs
    qp, qt, qh = _heads("q", q, qs)
    qop, qot, qoh = _heads("q_out", q_out, qs)
    hk, kp, kt, kh, kop, kot, koh = 0, None, 0, 0, None, 0, 0
    if k is not None:
        hk = ks[1]
        kp, kt, kh = _heads("k", k, ks)
        kop, kot, koh = _heads("k_out", k_out, ks)
    c = HeadNorm(T, hq, hk, D, rot, bool(interleaved), eps, rows, qt, qh, kt, kh, qot, qoh, kot, koh)
    _check("moe_head_norm_rotary", lib().moe_head_norm_rotary(
        ctypes.byref(c), qp, kp, _rows("w_q", w_q, chan, _BF16),
        _rows("w_k", w_k, chan, _BF16, k is None), _at(table, f32),
        _at(pos, i32), qop, kop, _at(status, i32), _stream(stream)))


def head_norm_rotary_workspace(T, hq, hk, D) -> int:
    """Scratch bytes of head_norm_rotary_backward."""
    v = ctypes.c_int64()
    _check("moe_head_norm_rotary_workspace",
           lib().moe_head_norm_rotary_workspace(T, hq, hk, D, ctypes.byref(v)))
    return v.value


def head_norm_rotary_backward(dq, dk, q, k, w_q, w_k, table, pos, dq_out, dk_out, dw_q, dw_k, ws,
                              status, eps=1e-6, interleaved=False, stream=None):
    """Gradients of head_norm_rotary for dq, dk (of q_out, k_out), from the
    forward's q and k: dq_out, dk_out (each may be its dq, dk or q, k), dw_q,
    dw_k [D] fp32.  None exactly where the forward's tensor is."""
    qs, ks, chan, rot, rows = _head_norm_shapes(q, k, table, pos)
    T, hq, D = qs
    none = k is None
    qp, qt, qh = _heads("q", q, qs)
    dqp, dqt, dqh = _heads("dq", dq, qs)
    qop, qot, qoh = _heads("dq_out", dq_out, qs)
    hk, kp, kt, kh, dkp, dkt, dkh, kop, kot, koh = 0, None, 0, 0, None, 0, 0, None, 0, 0
    if not none:
        hk = ks[1]
        kp, kt, kh = _heads("k", k, ks)
        dkp, dkt, dkh = _heads("dk", dk, ks)
        kop, kot, koh = _heads("dk_out", dk_out, ks)
    c = HeadNorm(T, hq, hk, D, rot, bool(interleaved), eps, rows, qt, qh, kt, kh, qot, qoh, kot, koh,
                 dqt, dqh, dkt, dkh)
    _check("moe_head_norm_rotary_backward", lib().moe_head_norm_rotary_backward(
        ctypes.byref(c), dqp, dkp, qp, kp, _rows("w_q", w_q, chan, _BF16),
        _rows("w_k", w_k, chan, _BF16, none), _at(table, f32),
        _at(pos, i32), qop, kop, _rows("dw_q", dw_q, chan, _F32),
        _rows("dw_k", dw_k, chan, _F32, none), _at(ws, u8), ws.numel(), _at(status, i32),
        _stream(stream)))


# ---------------------------------------------------------------- choice of experts

ROUTING_SCORES = {"softmax": 0, "sigmoid": 1}


class Routing:
    """A rule by which tokens choose top_k of n_experts (moe_routing_t): scores
    (softmax or sigmoid of the logits) and a bias for the choice alone, the best
    groups_kept of n_groups groups (by their group_top largest), the largest of
    those; weights renormalised over the chosen (renorm) and scaled."""

    def __init__(self, n_experts, top_k, score="softmax", n_groups=1, groups_kept=None,
                 group_top=1, renorm=True, scale=1.0):
        if score not in ROUTING_SCORES:
            raise ValueError(f"score must be one of {sorted(ROUTING_SCORES)}")
        self.n_experts, self.top_k = n_experts, top_k
        self.score, self.n_groups, self.group_top = ROUTING_SCORES[score], n_groups, group_top
        self.groups_kept = n_groups if groups_kept is None else groups_kept
        self.renorm, self.scale = bool(renorm), float(scale)

    def config(self, T, grad_f32=False) -> RoutingConfig:
        return RoutingConfig(T, self.n_experts, self.top_k, self.score, self.n_groups,
                             self.groups_kept, self.group_top, self.renorm, self.scale, grad_f32)


def _routing_shapes(routing, logits):
    if logits.dim() != 2:
        raise ValueError("logits is [T, experts]")
    T = logits.shape[0]
    return (T, routing.n_experts), (T, routing.top_k)


def router_select(routing, logits, bias, idx, w, stream=None):
    """idx [T, top_k] int32, w [T, top_k] fp32: the experts that the rule chooses
    for logits [T, n_experts] fp32 and bias [n_experts] fp32 (or None), in
    falling order of score + bias, and their weights."""
    rows, chosen = _routing_shapes(routing, logits)
    c = routing.config(rows[0])
    _check("moe_router_select", lib().moe_router_select(
        ctypes.byref(c), _rows("logits", logits, rows, _F32),
        _rows("bias", bias, rows[1:], _F32, True), _rows("idx", idx, chosen, _I32),
        _rows("w", w, chosen, _F32), _stream(stream)))


def router_select_backward(routing, logits, idx, dw, dlogits, stream=None):
    """dlogits [T, n_experts] (bf16 or fp32): gradient of router_select's logits
    for dw [T, top_k] fp32 of its weights; idx as the forward gave it."""
    rows, chosen = _routing_shapes(routing, logits)
    c = routing.config(rows[0], dlogits.dtype == f32)
    _check("moe_router_select_backward", lib().moe_router_select_backward(
        ctypes.byref(c), _rows("logits", logits, rows, _F32), _rows("idx", idx, chosen, _I32),
        _rows("dw", dw, chosen, _F32), _rows("dlogits", dlogits, rows, _RES), _stream(stream)))


# ---------------------------------------------------------------- embedding

def _embedding_config(table, out, T, scale, accumulate=False):
    if table.dim() != 2:
        raise ValueError("the table is [V, d]")
    V, d = table.shape
    return EmbeddingConfig(T, V, d, table.dtype == f32, out.dtype == f32, bool(accumulate), scale)


def embedding(table, ids, out, status, scale=1.0, stream=None):
    """out[t] = scale * table[ids[t]]: table [V, d], out [T, d], bf16 or fp32
    each, ids [T] int32; -1 (padding) gives zeros."""
    T = ids.numel()
    c = _embedding_config(table, out, T, scale)
    _check("moe_embedding", lib().moe_embedding(
        ctypes.byref(c), _rows("table", table, (c.V, c.d), _RES), _rows("ids", ids, (T,), _I32),
        _rows("out", out, (T, c.d), _RES), _at(status, i32), _stream(stream)))


class EmbeddingPlan:
    """The tokens of one batch by word, for embedding_backward: made from ids [T]
    int32 on the device, on the stream.  It serves any number of gradients of
    this T, vocab and d, one after another (it holds their scratch); refill()
    takes another batch's ids.  ``status`` receives MOE_EINVAL for ids outside
    the vocabulary other than -1; none of them has a gradient."""

    def __init__(self, ids, vocab, d, status=None, stream=None):
        if ids.dim() != 1:
            raise ValueError("ids is [T]")
        self.T, self.vocab, self.d = ids.numel(), vocab, d
        pb = ctypes.c_int64()
        _check("moe_embedding_workspace", lib().moe_embedding_workspace(
            self.T, vocab, d, ctypes.byref(pb)))
        with on_stream(stream):
            self.status = (torch.zeros(1, dtype=i32, device=ids.device) if status is None
                           else status)
            self.plan = torch.empty(pb.value, dtype=u8, device=ids.device)
        self.refill(ids, stream)

    def refill(self, ids, stream=None):
        _check("moe_embedding_plan", lib().moe_embedding_plan(
            self.T, self.vocab, self.d, _rows("ids", ids, (self.T,), _I32), _at(self.plan, u8),
            self.plan.numel(), _at(self.status, i32), _stream(stream)))


def embedding_backward(plan, dout, dtable, scale=1.0, accumulate=False, stream=None):
    """dtable[v] = scale * the sum of dout[t] over the plan's tokens of word v, in
    their order; dout [T, d], dtable [vocab, d], bf16 or fp32 each.  Words that do
    not occur become 0; accumulate: the sums are added to dtable instead."""
    c = _embedding_config(dtable, dout, plan.T, scale, accumulate)
    _check("moe_embedding_backward", lib().moe_embedding_backward(
        ctypes.byref(c), plan.plan.data_ptr(), plan.plan.numel(),
        _rows("dout", dout, (plan.T, plan.d), _RES),
        _rows("dtable", dtable, (plan.vocab, plan.d), _RES), _stream(stream)))


# ---------------------------------------------------------------- distillation loss

def _logits(name, t, shape, dtype):
    """(address, row stride) of [T, V] logits whose rows are contiguous."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: device tensor with contiguous rows required")
    return t.data_ptr(), t.stride(0)


def _distill_args(logits, ids, teacher, dlogits, temperature, scale):
    """(configuration, addresses of logits and dlogits, shapes of entries and tokens)."""
    zs, given, dt = logits.shape, ids.shape, logits.dtype
    if len(zs) != 2 or len(given) != 2 or dt not in _RES:
        raise ValueError("logits is [T, V] bf16 or fp32, ids [T, K]")
    T, V = zs
    K = given[1]
    zp, z_ld = _logits("logits", logits, zs, dt)
    dp, dz_ld = (None, 0) if dlogits is None else _logits("dlogits", dlogits, zs, dt)
    c = Distill(T, V, z_ld, dz_ld, K, dt == f32, teacher.dtype == f32, temperature, scale)
    return c, zp, dp, (T, K), (T,)


def distill_loss(logits, ids, teacher, weight, loss, lse, status, total=None, dlogits=None,
                 temperature=1.0, scale=1.0, stream=None):
    """loss[t] = scale weight[t] temperature^2 KL(teacher || student), the teacher
    given by its logits teacher [T, K] (bf16 or fp32) of the words ids [T, K] int32
    (-1: no entry), the student by logits [T, V] (bf16 or fp32, rows may be
    strided), both at that temperature; weight [T] fp32 or None.  loss, lse [T]
    fp32; total [1] fp32 receives the losses' sum, dlogits (may be logits) their
    gradient in the same pass.  Rows without weight or entries have loss 0."""
    c, zp, dp, given, tok = _distill_args(logits, ids, teacher, dlogits, temperature, scale)
    _check("moe_distill_loss", lib().moe_distill_loss(
        ctypes.byref(c), zp, _rows("ids", ids, given, _I32), _rows("teacher", teacher, given, _RES),
        _rows("weight", weight, tok, _F32, True), _rows("loss", loss, tok, _F32),
        _rows("lse", lse, tok, _F32), _rows("total", total, (1,), _F32, True), dp,
        _at(status, i32), _stream(stream)))


def distill_loss_backward(logits, ids, teacher, weight, lse, dlogits, status, temperature=1.0,
                          scale=1.0, stream=None):
    """dlogits (may be logits): gradient of distill_loss's summed loss, from the
    forward's inputs and lse."""
    if dlogits is None:
        raise ValueError("dlogits: tensor required")
    c, zp, dp, given, tok = _distill_args(logits, ids, teacher, dlogits, temperature, scale)
    _check("moe_distill_loss_backward", lib().moe_distill_loss_backward(
        ctypes.byref(c), zp, _rows("ids", ids, given, _I32), _rows("teacher", teacher, given, _RES),
        _rows("weight", weight, tok, _F32, True), _rows("lse", lse, tok, _F32), dp,
        _at(status, i32), _stream(stream)))
