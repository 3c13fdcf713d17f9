"""ctypes binding of libdsa.so.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Functions take torch CUDA tensors, check dtype, device and layout,
pass raw pointers and the current CUDA stream, and raise DsaError on a
non-zero status.  Importing this module without the built library raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

DSA_OK = 0
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "workspace missing or too small",
          4: "CUDA error", 5: "device wait timed out"}
DEVERR_POSITION, DEVERR_PAGE, DEVERR_TIMEOUT, DEVERR_SHAPE = 1, 2, 4, 8
MODE_PREFILL, MODE_DECODE = 0, 1


class DsaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {STATUS.get(status, status)} (status {status})")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"libdsa.so is not built ({LIB_PATH}); run long_context_sparse_02_b200/build.py")

lib = ctypes.CDLL(LIB_PATH)

P = ctypes.c_void_p
I32 = ctypes.c_int32
I64 = ctypes.c_int64
SZ = ctypes.c_size_t
F32 = ctypes.c_float


class Paged(ctypes.Structure):
    _fields_ = [("seq_lens", P), ("block_table", P), ("num_seqs", I32), ("max_blocks_per_seq", I32),
                ("page_size", I32), ("num_pages", I32)]


class LayerArgs(ctypes.Structure):
    _fields_ = [("mode", I32), ("q_idx", P), ("w", P), ("k_idx_cache", P), ("q", P), ("kv_cache", P),
                ("gate", P), ("pg", Paged), ("q_seq", P), ("q_pos", P), ("T", I32), ("HI", I32), ("DI", I32),
                ("K", I32), ("H", I32), ("Dqk", I32), ("Dv", I32), ("max_len", I32), ("sm_scale", F32),
                ("out", P), ("idx_out", P), ("lse", P), ("q_idx_scales", P), ("k_idx_scales", P)]


class RopeSpec(ctypes.Structure):
    _fields_ = [("inv_freq", P), ("dim", I32), ("offset", I32), ("layout", I32), ("inverse", I32), ("factor", F32)]


class KvCache(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("k_page_stride", I64), ("k_row_stride", I64), ("k_head_stride", I64),
                ("v_page_stride", I64), ("v_row_stride", I64), ("v_head_stride", I64), ("heads", I32), ("Dk", I32),
                ("Dv", I32), ("dtype", I32), ("k_scale", F32), ("v_scale", F32)]


lib.dsa_abi_version.restype = I32
lib.dsa_abi_version.argtypes = []
lib.dsa_status_string.restype = ctypes.c_char_p
lib.dsa_status_string.argtypes = [ctypes.c_int]
lib.dsa_device_error.restype = ctypes.c_int
lib.dsa_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32), I32]
lib.dsa_indexer_scores.restype = ctypes.c_int
lib.dsa_indexer_scores.argtypes = [P, P, P, ctypes.POINTER(Paged), P, P, I32, I32, I32, I32, P, I64, P]
lib.dsa_indexer_scores_mx.restype = ctypes.c_int
lib.dsa_indexer_scores_mx.argtypes = [P, P, P, P, P, ctypes.POINTER(Paged), P, P, I32, I32, I32, I32, P, I64, P]
lib.dsa_append_kv_mx.restype = ctypes.c_int
lib.dsa_append_kv_mx.argtypes = [P, P, P, P, ctypes.POINTER(Paged), I32, I32, I32, P, P, P, P]
lib.dsa_topk_workspace_bytes.restype = SZ
lib.dsa_topk_workspace_bytes.argtypes = [I32, I32, I32]
lib.dsa_topk.restype = ctypes.c_int
lib.dsa_topk.argtypes = [P, I64, P, I32, I32, I32, P, P, SZ, P]
lib.dsa_topk_hist_workspace_bytes.restype = SZ
lib.dsa_topk_hist_workspace_bytes.argtypes = [I32, I32]
lib.dsa_topk_hist.restype = ctypes.c_int
lib.dsa_topk_hist.argtypes = [P, I64, P, I32, I32, I32, P, P, P, SZ, P]
lib.dsa_topk_static.restype = ctypes.c_int
lib.dsa_topk_static.argtypes = [P, I64, P, I32, I32, I32, P, P]
lib.dsa_sparse_attn_workspace_bytes.restype = SZ
lib.dsa_sparse_attn_workspace_bytes.argtypes = [I32, I32, I32, I32]
lib.dsa_sparse_attn.restype = ctypes.c_int
lib.dsa_sparse_attn.argtypes = [P, P, ctypes.POINTER(Paged), P, P, I32, P, F32, I32, I32, I32, I32, P, P, P,
                                SZ, P]
lib.dsa_layer_workspace_bytes.restype = SZ
lib.dsa_layer_workspace_bytes.argtypes = [ctypes.POINTER(LayerArgs)]
lib.dsa_layer_forward.restype = ctypes.c_int
lib.dsa_layer_forward.argtypes = [ctypes.POINTER(LayerArgs), P, SZ, P]
lib.dsa_layer_forward_profiled.restype = ctypes.c_int
lib.dsa_layer_forward_profiled.argtypes = [ctypes.POINTER(LayerArgs), P, SZ, ctypes.POINTER(P), P]
lib.dsa_layer_kernel_launches.restype = I32
lib.dsa_append_kv.restype = ctypes.c_int
lib.dsa_append_kv.argtypes = [P, F32, P, P, P, ctypes.POINTER(Paged), I32, I32, I32, P, P, P]
lib.dsa_layer_kernel_launches.argtypes = [ctypes.POINTER(LayerArgs)]
lib.dsa_cp_candidates.restype = ctypes.c_int
lib.dsa_cp_candidates.argtypes = [P, I64, P, I32, I32, P, P, P, P]
lib.dsa_cp_select_workspace_bytes.restype = SZ
lib.dsa_cp_select_workspace_bytes.argtypes = [I32, I32, I32]
lib.dsa_cp_select.restype = ctypes.c_int
lib.dsa_cp_select.argtypes = [P, P, I32, I32, I32, P, P, P, P, P, SZ, P]
lib.dsa_cp_lse_merge.restype = ctypes.c_int
lib.dsa_cp_lse_merge.argtypes = [P, P, I32, I32, I32, I32, P, P]
lib.dsa_test_skip_indexer_tile.restype = ctypes.c_int
lib.dsa_test_skip_indexer_tile.argtypes = [I64]
lib.dsa_swa_decode.restype = ctypes.c_int
lib.dsa_swa_decode.argtypes = [P, P, P, P, I32, I32, I32, I32, F32, P, P]
lib.dsa_rope_frequencies.restype = ctypes.c_int
lib.dsa_rope_frequencies.argtypes = [I32, ctypes.c_double, I32, ctypes.c_double, I32, ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(F32)]
lib.dsa_rope.restype = ctypes.c_int
# (structs of the calls below by address: see _addr)
lib.dsa_rope.argtypes = [P, I64, I64, I32, P, I64, I64, P, I64, I64, I32, P, I64, I64, P, I32, I32, I32, P, P]
lib.dsa_append_rope.restype = ctypes.c_int
lib.dsa_append_rope.argtypes = [P, I64, I64, P, I64, I64, P, I64, I64, I32, P, I64, I64, P, P, P, I32, I32, P, P, P]
lib.dsa_paged_attn_workspace_bytes.restype = SZ
lib.dsa_paged_attn_workspace_bytes.argtypes = [I32, I32, I32, ctypes.POINTER(KvCache), I32, I32, I32]
lib.dsa_paged_attn.restype = ctypes.c_int
lib.dsa_paged_attn.argtypes = [P, I64, I64, I32, P, P, P, I32, I32, I32, I32, F32, I32, P, P, P, SZ, P]

EXPORTS = ["dsa_abi_version", "dsa_status_string", "dsa_device_error", "dsa_indexer_scores", "dsa_indexer_scores_mx",
           "dsa_append_kv_mx",
           "dsa_topk_workspace_bytes", "dsa_topk", "dsa_topk_hist_workspace_bytes", "dsa_topk_hist", "dsa_topk_static", "dsa_sparse_attn_workspace_bytes",
           "dsa_sparse_attn",
           "dsa_layer_workspace_bytes", "dsa_layer_forward", "dsa_layer_forward_profiled",
           "dsa_layer_kernel_launches", "dsa_swa_decode", "dsa_append_kv", "dsa_cp_candidates",
           "dsa_cp_select_workspace_bytes", "dsa_cp_select", "dsa_cp_lse_merge",
           "dsa_test_skip_indexer_tile", "dsa_rope_frequencies", "dsa_rope", "dsa_append_rope",
           "dsa_paged_attn_workspace_bytes", "dsa_paged_attn"]


def _check(fn: str, status: int):
    if status != DSA_OK:
        raise DsaError(fn, status)


def _ptr(t, dtype, name, nullable=False):
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def paged(seq_lens: torch.Tensor, block_table: torch.Tensor, num_pages: int, page_size: int = 64) -> Paged:
    """The C struct holds raw pointers, so it also keeps the two tensors alive."""
    if seq_lens.dim() != 1 or block_table.dim() != 2 or block_table.shape[0] < seq_lens.shape[0]:
        raise ValueError(f"block_table must have a row for each of seq_lens, got {tuple(block_table.shape)} for "
                         f"{tuple(seq_lens.shape)}")
    pg = Paged(_ptr(seq_lens, torch.int32, "seq_lens"), _ptr(block_table, torch.int32, "block_table"),
               int(seq_lens.shape[0]), int(block_table.shape[1]), int(page_size), int(num_pages))
    pg._tensors = (seq_lens, block_table)
    return pg


def device_error(reset: bool = True) -> int:
    code = ctypes.c_uint32(0)
    _check("dsa_device_error", lib.dsa_device_error(ctypes.byref(code), 1 if reset else 0))
    return int(code.value)


def indexer_scores(q_idx, w, k_cache, pg: Paged, q_seq, q_pos, max_len: int, scores):
    """q_idx uint8 [T,HI,DI]; w fp32 [T,HI]; k_cache uint8 [pages,64,DI];
    q_seq/q_pos int32 [T] or None (decode); scores fp32 [T, ld]."""
    T, HI, DI = q_idx.shape
    _check("dsa_indexer_scores", lib.dsa_indexer_scores(
        _ptr(q_idx, torch.uint8, "q_idx"), _ptr(w, torch.float32, "w"), _ptr(k_cache, torch.uint8, "k_cache"),
        ctypes.byref(pg), _ptr(q_seq, torch.int32, "q_seq", True), _ptr(q_pos, torch.int32, "q_pos", True),
        T, HI, DI, int(max_len), _ptr(scores, torch.float32, "scores"), int(scores.shape[1]), _stream()))
    return scores


def topk_workspace_bytes(R: int, K: int, max_row_len: int) -> int:
    return int(lib.dsa_topk_workspace_bytes(R, K, max_row_len))


def topk(scores, row_len, K: int, max_row_len: int, idx=None, ws=None):
    R, ld = scores.shape
    if idx is None:
        idx = torch.empty((R, K), dtype=torch.int32, device=scores.device)
    need = topk_workspace_bytes(R, K, max_row_len)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=scores.device)
    _check("dsa_topk", lib.dsa_topk(
        _ptr(scores, torch.float32, "scores"), ld, _ptr(row_len, torch.int32, "row_len"), R, K, int(max_row_len),
        _ptr(idx, torch.int32, "idx"), _ptr(ws, torch.uint8, "ws", True), need if ws is None else ws.numel(),
        _stream()))
    return idx


def topk_hist(scores, row_len, hist, K: int, max_row_len: int, idx=None, ws=None):
    """hist uint32 (as torch.int32) [R, 2048]: counts of key(score) >> 21 per row; zeroed by the call."""
    R, ld = scores.shape
    if idx is None:
        idx = torch.empty((R, K), dtype=torch.int32, device=scores.device)
    need = int(lib.dsa_topk_hist_workspace_bytes(R, int(max_row_len)))
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=scores.device)
    _check("dsa_topk_hist", lib.dsa_topk_hist(
        _ptr(scores, torch.float32, "scores"), ld, _ptr(row_len, torch.int32, "row_len"), R, K, int(max_row_len),
        _ptr(hist, torch.int32, "hist"), _ptr(idx, torch.int32, "idx"), _ptr(ws, torch.uint8, "ws"), ws.numel(),
        _stream()))
    return idx


def sparse_attn_workspace_bytes(T: int, H: int, K: int, Dv: int) -> int:
    return int(lib.dsa_sparse_attn_workspace_bytes(T, H, K, Dv))


def sparse_attn(q, kv_cache, pg: Paged, q_seq, idx, gate, sm_scale: float, Dv: int, out=None, lse=None, ws=None):
    """q bf16 [T,H,Dqk]; kv_cache bf16 [pages,64,Dqk]; idx int32 [T,K]; gate bf16 [T,H]."""
    T, H, Dqk = q.shape
    K = idx.shape[1]
    if out is None:
        out = torch.empty((T, H, Dv), dtype=torch.bfloat16, device=q.device)
    need = sparse_attn_workspace_bytes(T, H, K, Dv)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check("dsa_sparse_attn", lib.dsa_sparse_attn(
        _ptr(q, torch.bfloat16, "q"), _ptr(kv_cache, torch.bfloat16, "kv_cache"), ctypes.byref(pg),
        _ptr(q_seq, torch.int32, "q_seq", True), _ptr(idx, torch.int32, "idx"), K,
        _ptr(gate, torch.bfloat16, "gate"), float(sm_scale), T, H, Dqk, Dv, _ptr(out, torch.bfloat16, "out"),
        _ptr(lse, torch.float32, "lse", True), _ptr(ws, torch.uint8, "ws", True),
        need if ws is None else ws.numel(), _stream()))
    return out


def layer_args(mode, q_idx, w, k_cache, q, kv_cache, gate, pg: Paged, q_seq, q_pos, K: int, Dv: int,
               sm_scale: float, max_len: int, out, idx_out=None, lse=None, q_scales=None,
               k_scales=None) -> LayerArgs:
    T, HI, DI = q_idx.shape
    _, H, Dqk = q.shape
    a = LayerArgs(int(mode), _ptr(q_idx, torch.uint8, "q_idx"), _ptr(w, torch.float32, "w"),
                     _ptr(k_cache, torch.uint8, "k_cache"), _ptr(q, torch.bfloat16, "q"),
                     _ptr(kv_cache, torch.bfloat16, "kv_cache"), _ptr(gate, torch.bfloat16, "gate"), pg,
                     _ptr(q_seq, torch.int32, "q_seq", True), _ptr(q_pos, torch.int32, "q_pos", True),
                     T, HI, DI, int(K), H, Dqk, int(Dv), int(max_len), float(sm_scale),
                     _ptr(out, torch.bfloat16, "out"), _ptr(idx_out, torch.int32, "idx_out", True),
                     _ptr(lse, torch.float32, "lse", True), _ptr(q_scales, torch.uint8, "q_scales", True),
                     _ptr(k_scales, torch.uint8, "k_scales", True))
    a._tensors = (q_idx, w, k_cache, q, kv_cache, gate, getattr(pg, "_tensors", None), q_seq, q_pos, out, idx_out,
                  lse, q_scales, k_scales)
    return a


def layer_workspace_bytes(args: LayerArgs) -> int:
    return int(lib.dsa_layer_workspace_bytes(ctypes.byref(args)))


def layer_kernel_launches(args: LayerArgs) -> int:
    return int(lib.dsa_layer_kernel_launches(ctypes.byref(args)))


def layer_forward(args: LayerArgs, ws: torch.Tensor):
    _check("dsa_layer_forward", lib.dsa_layer_forward(ctypes.byref(args), _ptr(ws, torch.uint8, "ws"),
                                                      ws.numel(), _stream()))


def layer_forward_profiled(args: LayerArgs, ws: torch.Tensor, events):
    """events: four recorded-once torch.cuda.Event objects (or None)."""
    arr = (P * 4)(*[P(e.cuda_event) if e is not None else P(0) for e in events])
    _check("dsa_layer_forward_profiled", lib.dsa_layer_forward_profiled(
        ctypes.byref(args), _ptr(ws, torch.uint8, "ws"), ws.numel(), arr, _stream()))


def swa_decode(q, k_ring, v_ring, seq_lens, window: int, sm_scale: float, out=None):
    B, H, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    _check("dsa_swa_decode", lib.dsa_swa_decode(
        _ptr(q, torch.bfloat16, "q"), _ptr(k_ring, torch.bfloat16, "k_ring"), _ptr(v_ring, torch.bfloat16, "v_ring"),
        _ptr(seq_lens, torch.int32, "seq_lens"), B, H, D, int(window), float(sm_scale),
        _ptr(out, torch.bfloat16, "out"), _stream()))
    return out


def append_kv(k_new, k_scale: float, latent_new, tok_seq, tok_pos, pg: Paged, k_cache, kv_cache):
    """k_new bf16 [n, DI]; latent_new bf16 [n, Dqk] or None; tok_seq/tok_pos int32 [n];
    k_cache uint8 (e4m3) [pages, 64, DI] and kv_cache bf16 [pages, 64, Dqk], written in place."""
    n, DI = k_new.shape
    Dqk = int(kv_cache.shape[-1]) if kv_cache is not None else 0
    _check("dsa_append_kv", lib.dsa_append_kv(
        _ptr(k_new, torch.bfloat16, "k_new"), float(k_scale), _ptr(latent_new, torch.bfloat16, "latent_new", True),
        _ptr(tok_seq, torch.int32, "tok_seq"), _ptr(tok_pos, torch.int32, "tok_pos"), ctypes.byref(pg), n, DI, Dqk,
        _ptr(k_cache, torch.uint8, "k_cache"), _ptr(kv_cache, torch.bfloat16, "kv_cache", True), _stream()))


def cp_candidates(scores, idx_local, lo, cand_score=None, cand_pos=None):
    """(score, global position) of each locally kept index; scores fp32 [B, ld], idx_local int32 [B, K]."""
    B, K = idx_local.shape
    if cand_score is None:
        cand_score = torch.empty((B, K), dtype=torch.float32, device=scores.device)
    if cand_pos is None:
        cand_pos = torch.empty((B, K), dtype=torch.int32, device=scores.device)
    _check("dsa_cp_candidates", lib.dsa_cp_candidates(
        _ptr(scores, torch.float32, "scores"), int(scores.shape[1]), _ptr(idx_local, torch.int32, "idx_local"), B, K,
        _ptr(lo, torch.int32, "lo"), _ptr(cand_score, torch.float32, "cand_score"),
        _ptr(cand_pos, torch.int32, "cand_pos"), _stream()))
    return cand_score, cand_pos


def cp_select(cand_score, cand_pos, lo, hi, idx_global=None, idx_local=None, ws=None):
    """cand_score fp32 / cand_pos int32 [G, B, K] (every rank's candidates) -> (idx_global, idx_local) [B, K]."""
    G, B, K = cand_score.shape
    dev = cand_score.device
    if idx_global is None:
        idx_global = torch.empty((B, K), dtype=torch.int32, device=dev)
    if idx_local is None:
        idx_local = torch.empty((B, K), dtype=torch.int32, device=dev)
    need = int(lib.dsa_cp_select_workspace_bytes(G, B, K))
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _check("dsa_cp_select", lib.dsa_cp_select(
        _ptr(cand_score, torch.float32, "cand_score"), _ptr(cand_pos, torch.int32, "cand_pos"), G, B, K,
        _ptr(lo, torch.int32, "lo"), _ptr(hi, torch.int32, "hi"), _ptr(idx_global, torch.int32, "idx_global"),
        _ptr(idx_local, torch.int32, "idx_local"), _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream()))
    return idx_global, idx_local


def cp_lse_merge(o, lse, out=None):
    """o bf16 [G, B, H, Dv], lse fp32 [G, B, H] -> out bf16 [B, H, Dv]."""
    G, B, H, Dv = o.shape
    if out is None:
        out = torch.empty((B, H, Dv), dtype=torch.bfloat16, device=o.device)
    _check("dsa_cp_lse_merge", lib.dsa_cp_lse_merge(
        _ptr(o, torch.bfloat16, "o"), _ptr(lse, torch.float32, "lse"), G, B, H, Dv, _ptr(out, torch.bfloat16, "out"),
        _stream()))
    return out


def indexer_scores_mx(q_idx, q_scales, w, k_cache, k_scales, pg: Paged, q_seq, q_pos, max_len: int, scores):
    """MXFP8 indexer: q_idx uint8 [T,HI,DI] and q_scales uint8 [T,HI,DI/32]; k_cache uint8 [pages,64,DI] and
    k_scales uint8 [pages,64,DI/32]; w fp32 [T,HI]; scores fp32 [T, ld]."""
    T, HI, DI = q_idx.shape
    _check("dsa_indexer_scores_mx", lib.dsa_indexer_scores_mx(
        _ptr(q_idx, torch.uint8, "q_idx"), _ptr(q_scales, torch.uint8, "q_scales"), _ptr(w, torch.float32, "w"),
        _ptr(k_cache, torch.uint8, "k_cache"), _ptr(k_scales, torch.uint8, "k_scales"), ctypes.byref(pg),
        _ptr(q_seq, torch.int32, "q_seq", True), _ptr(q_pos, torch.int32, "q_pos", True), T, HI, DI, int(max_len),
        _ptr(scores, torch.float32, "scores"), int(scores.shape[1]), _stream()))
    return scores


def append_kv_mx(k_new, latent_new, tok_seq, tok_pos, pg: Paged, k_cache, k_scales, kv_cache):
    """MXFP8 append: k_new bf16 [n, DI]; latent_new bf16 [n, Dqk] or None; k_cache uint8 [pages, 64, DI],
    k_scales uint8 [pages, 64, DI/32] and kv_cache bf16 [pages, 64, Dqk], written in place."""
    n, DI = k_new.shape
    Dqk = int(kv_cache.shape[-1]) if kv_cache is not None else 0
    _check("dsa_append_kv_mx", lib.dsa_append_kv_mx(
        _ptr(k_new, torch.bfloat16, "k_new"), _ptr(latent_new, torch.bfloat16, "latent_new", True),
        _ptr(tok_seq, torch.int32, "tok_seq"), _ptr(tok_pos, torch.int32, "tok_pos"), ctypes.byref(pg), n, DI, Dqk,
        _ptr(k_cache, torch.uint8, "k_cache"), _ptr(k_scales, torch.uint8, "k_scales"),
        _ptr(kv_cache, torch.bfloat16, "kv_cache", True), _stream()))


# ---- rotary positions, the rotating append and attention over a paged K/V cache ----------------------------------

BF16, F16, E4M3 = 0, 1, 2
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_SCHEMES = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}
_IO = {torch.bfloat16: BF16, torch.float16: F16}
_CACHE = {torch.bfloat16: BF16, torch.float16: F16, torch.uint8: E4M3, torch.float8_e4m3fn: E4M3}


# These calls are made once a layer and step: the checks read each tensor's facts once and the arguments go over as
# plain integers (a decode step's rotation took 17 us of host time otherwise, most of it spent on wrappers).
_raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream().cuda_stream without the Stream object


def _device(t, name: str) -> int:
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return d


def _on(dev: int, name: str, t):
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


def _call(fn: str, f, dev: int, *args):
    """The library call on device dev's current stream, with that device current."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            _check(fn, f(*args, torch.cuda.current_stream().cuda_stream))
    else:
        status = f(*args, _raw_stream(dev))
        if status:
            raise DsaError(fn, status)


def _addr(struct) -> int:
    return ctypes.addressof(struct)


def _heads(t, name: str, dev: int, dtype, shape):
    """[tokens, heads, width] with a contiguous last dimension: (pointer, token stride, head stride)."""
    if t.get_device() != dev or t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} tensor {tuple(shape)} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}")
    ts, hs, ds = t.stride()
    if ds != 1 and shape[2] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr(), ts, hs


def _first(t, name: str):
    """(device, dtype, tokens, heads, width) of the tensor that the others of a call go by."""
    dev = _device(t, name)
    if t.dim() != 3 or t.dtype not in _IO:
        raise ValueError(f"{name} must be a bf16 or fp16 tensor [tokens, heads, width], got {t.dtype} {tuple(t.shape)}")
    return (dev, t.dtype, *t.shape)


def _tokens(t, name: str, dev: int, n: int) -> int:
    if t.get_device() != dev or t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries on cuda:{dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def rope_frequencies(dim: int, base: float = 10000.0, scheme: str = "plain", scale: float = 1.0, orig_len: int = 0):
    """(inverse frequencies, a CPU fp64 tensor [dim/2]; factor): scheme "plain", "linear", "ntk" or "yarn" for contexts
    `scale` times as long as the `orig_len` of training."""
    if scheme not in ROPE_SCHEMES:
        raise ValueError(f"scheme must be one of {sorted(ROPE_SCHEMES)}")
    freq = torch.empty(max(int(dim) // 2, 1), dtype=torch.float64)
    factor = F32(1.0)
    _check("dsa_rope_frequencies", lib.dsa_rope_frequencies(
        int(dim), float(base), ROPE_SCHEMES[scheme], float(scale), int(orig_len),
        ctypes.cast(freq.data_ptr(), ctypes.POINTER(ctypes.c_double)), ctypes.byref(factor)))
    return freq, float(factor.value)


def rope_spec(inv_freq: torch.Tensor, offset: int = 0, interleaved: bool = False, inverse: bool = False,
              factor: float = 1.0) -> RopeSpec:
    """inv_freq fp64 [dim/2] on the GPU; elements offset .. offset + dim of each head are rotated.  `inverse` is the
    transpose, a gradient's way back; to undo a rotation of some factor, give the inverse 1 / factor.  Keeps inv_freq alive."""
    spec = RopeSpec(_ptr(inv_freq, torch.float64, "inv_freq"), 2 * int(inv_freq.numel()), int(offset),
                    ROPE_INTERLEAVED if interleaved else ROPE_HALF, int(bool(inverse)), float(factor))
    spec._tensors = (inv_freq,)
    spec._device = inv_freq.get_device()
    return spec


def kv_cache(k: torch.Tensor, v: torch.Tensor = None, k_scale: float = 1.0, v_scale: float = 1.0) -> KvCache:
    """A paged cache [pages, 64, heads, width] of keys and (optionally) values: bf16, fp16, or e4m3 codes of value * scale
    (uint8 or float8_e4m3fn).  Any strides with a contiguous last dimension.  The sparse layer's latent cache
    [pages, 64, 576] is kv_cache(latents.unsqueeze(2)): append_rope then writes the latent rows, rotated, and append_kv,
    given no latent rows, the indexer keys alone.  Keeps both tensors alive."""
    for name, t in (("k", k), ("v", v)):
        if t is None:
            continue
        if not t.is_cuda or t.dim() != 4 or t.shape[1] != 64 or t.dtype not in _CACHE or t.stride(3) != 1:
            raise ValueError(f"{name} must be a CUDA tensor [pages, 64, heads, width] of bf16, fp16 or e4m3 codes with a "
                             f"contiguous last dimension, got {t.dtype} {tuple(t.shape)}")
        if t.dtype != k.dtype or t.shape[:3] != k.shape[:3] or t.device != k.device:
            raise ValueError("k and v must have the same dtype, device, pages and heads")
    sv = v.stride() if v is not None else (0, 0, 0)
    c = KvCache(k.data_ptr(), v.data_ptr() if v is not None else None, *k.stride()[:3], *sv[:3], int(k.shape[2]),
                int(k.shape[3]), int(v.shape[3]) if v is not None else 0, _CACHE[k.dtype], float(k_scale), float(v_scale))
    c._tensors = (k, v)
    c._device, c._pages = k.get_device(), int(k.shape[0])
    return c


def _cache_fits(cache: KvCache, pg: Paged, dev: int):
    if cache._pages < pg.num_pages:
        raise ValueError(f"the cache has {cache._pages} pages, the page table {pg.num_pages}")
    if cache._device != dev:
        raise ValueError(f"the cache must be on cuda:{dev}")
    _on(dev, "seq_lens", pg._tensors[0])
    _on(dev, "block_table", pg._tensors[1])


def _spec_fits(spec: RopeSpec, dev: int) -> int:
    if spec._device != dev:
        raise ValueError(f"inv_freq must be on cuda:{dev}")
    return ctypes.addressof(spec)


def rope(q, pos, spec: RopeSpec, k=None, q_out=None, k_out=None):
    """Rotary positions on q [T, H, D] and (optionally, in the same launch) k [T, Hk, D], bf16 or fp16, at pos int32 [T].
    q_out / k_out default to new dense tensors; pass q / k themselves to rotate in place.  Returns (q_out, k_out)."""
    dev, dtype, T, H, D = _first(q, "q")
    if q_out is None:
        q_out = q.new_empty((T, H, D))
    ka, ko, Hk = (None, 0, 0), (None, 0, 0), 0
    if k is not None:
        if k.dim() != 3:
            raise ValueError("k must be [tokens, heads, width]")
        Hk = k.shape[1]
        if k_out is None:
            k_out = k.new_empty((T, Hk, D))
        ka, ko = _heads(k, "k", dev, dtype, (T, Hk, D)), _heads(k_out, "k_out", dev, dtype, (T, Hk, D))
    _call("dsa_rope", lib.dsa_rope, dev, *_heads(q, "q", dev, dtype, (T, H, D)), H,
          *_heads(q_out, "q_out", dev, dtype, (T, H, D)), *ka, Hk, *ko, _tokens(pos, "pos", dev, T), T, D, _IO[dtype],
          _spec_fits(spec, dev))
    return q_out, k_out


def append_rope(k_new, v_new, tok_seq, tok_pos, pg: Paged, cache: KvCache, spec: RopeSpec = None, q=None, q_out=None):
    """k_new [n, heads, Dk] (rotated to tok_pos) and v_new [n, heads, Dv] or None into the cache; q [n, H, Dk], where given,
    rotated in the same launch into q_out (default: a new dense tensor; q itself for in place), which is returned."""
    dev, dtype, n, _, _ = _first(k_new, "k_new")
    _cache_fits(cache, pg, dev)
    heads, Dk = cache.heads, cache.Dk
    ka = _heads(k_new, "k_new", dev, dtype, (n, heads, Dk))
    va = (None, 0, 0) if v_new is None else _heads(v_new, "v_new", dev, dtype, (n, heads, cache.Dv))
    qa, qo, H = (None, 0, 0), (None, 0, 0), 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [tokens, heads, width]")
        H = q.shape[1]
        if q_out is None:
            q_out = q.new_empty((n, H, Dk))
        qa, qo = _heads(q, "q", dev, dtype, (n, H, Dk)), _heads(q_out, "q_out", dev, dtype, (n, H, Dk))
    _call("dsa_append_rope", lib.dsa_append_rope, dev, *ka, *va, *qa, H, *qo, _tokens(tok_seq, "tok_seq", dev, n),
          _tokens(tok_pos, "tok_pos", dev, n), _addr(pg), n, _IO[dtype], None if spec is None else _spec_fits(spec, dev),
          _addr(cache))
    return q_out if q is not None else None


def paged_attn_workspace(T: int, H: int, cache: KvCache, pg: Paged, max_q: int, max_len: int, window: int = 0):
    """A workspace for paged_attn calls of at most these sizes, on the cache's device."""
    dev = cache._tensors[0].device
    with torch.cuda.device(dev):
        need = int(lib.dsa_paged_attn_workspace_bytes(int(T), pg.num_seqs, int(H), ctypes.byref(cache), int(max_q),
                                                      int(max_len), int(window)))
        return torch.empty(max(need, 256), dtype=torch.uint8, device=dev)


def paged_attn(q, cache: KvCache, pg: Paged, q_start, max_q: int, max_len: int, window: int = 0, sm_scale: float = None,
               want_lse: bool = False, out=None, lse=None, ws=None):
    """Attention of q [T, H, D], each sequence's newest tokens (rows q_start[b] .. q_start[b+1], int32 [num_seqs + 1]; None:
    one each), over the paged cache, causal, optionally within a window.  Returns out, or (out, lse) with want_lse or lse."""
    dev, dtype, T, H, D = _first(q, "q")
    _cache_fits(cache, pg, dev)
    if D != cache.Dk:
        raise ValueError(f"q must have heads of {cache.Dk}, got {D}")
    if out is None:
        out = q.new_empty((T, H, D))
    elif out.get_device() != dev or out.dtype != dtype or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be dense, with q's shape, dtype and device")
    if lse is None:
        if want_lse:
            lse = q.new_empty((T, H), dtype=torch.float32)
    elif lse.get_device() != dev or lse.dtype != torch.float32 or lse.shape != (T, H) or not lse.is_contiguous():
        raise ValueError(f"lse must be a dense fp32 tensor [{T}, {H}] on cuda:{dev}")
    if ws is None:
        ws = paged_attn_workspace(T, H, cache, pg, max_q, max_len, window)
    elif ws.get_device() != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"ws must be a dense uint8 tensor on cuda:{dev}")
    _call("dsa_paged_attn", lib.dsa_paged_attn, dev, *_heads(q, "q", dev, dtype, (T, H, D)), H, _addr(cache), _addr(pg),
          None if q_start is None else _tokens(q_start, "q_start", dev, pg.num_seqs + 1), T, max_q, max_len, window,
          D ** -0.5 if sm_scale is None else sm_scale, _IO[dtype], out.data_ptr(), None if lse is None else lse.data_ptr(),
          ws.data_ptr(), ws.numel())
    return out if lse is None else (out, lse)
