"""Thin ctypes binding of libnq.so (include/nq.h).  Argument marshalling only:
every step of the hot path runs in the library's CUDA kernels.  PyTorch
provides device memory and the current stream.

The library must have been built (``quantized_self_speculative_gb300.build``);
there is no fallback: a missing library raises immediately.
"""
from __future__ import annotations

import ctypes as C
import os
import threading
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnq.so")

NQ_OK, NQ_ERR_ARG, NQ_ERR_SHAPE, NQ_ERR_ALIGN, NQ_ERR_CUDA = 0, 1, 2, 3, 4
NQ_ERR_NONFINITE, NQ_ERR_TIMEOUT, NQ_ERR_WORKSPACE, NQ_ERR_TOKEN = 5, 6, 7, 8
NQ_DEV_NONFINITE, NQ_DEV_BAD_TOKEN, NQ_DEV_TIMEOUT, NQ_DEV_ACT_RANGE, NQ_DEV_SEQ_FULL = 0x1, 0x2, 0x4, 0x8, 0x10
NQ_DEV_BAD_PAGE, NQ_DEV_POOL_FULL, NQ_DEV_BAD_TREE = 0x20, 0x40, 0x80
KV_NESTED44, KV_BF16 = 0, 1
FMT_NESTED44, FMT_INT4, FMT_FP8E4M3_ROW, FMT_FP16 = 0, 1, 2, 3

_lock = threading.Lock()
_lib = None


class NQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


class nq_weights(C.Structure):
    _fields_ = [("n_out", C.c_int32), ("k_in", C.c_int32), ("group", C.c_int32), ("format", C.c_int32),
                ("base", C.c_void_p), ("resid", C.c_void_p), ("scales", C.c_void_p)]


class nq_kv_cache(C.Structure):
    _fields_ = [("batch", C.c_int32), ("heads_kv", C.c_int32), ("head_dim", C.c_int32), ("group", C.c_int32),
                ("max_len", C.c_int32), ("pad", C.c_int32),
                ("k_base", C.c_void_p), ("k_resid", C.c_void_p), ("k_scales", C.c_void_p),
                ("v_base", C.c_void_p), ("v_resid", C.c_void_p), ("v_scales", C.c_void_p)]


class nq_rope_plan(C.Structure):
    _fields_ = [("rot_dim", C.c_int32), ("layout", C.c_int32), ("mscale", C.c_float), ("mscale_lo", C.c_float),
                ("rates", C.c_void_p)]


class nq_page_pool(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("layers", "n_pages", "page_size", "heads_kv", "head_dim", "group", "format",
                                         "pad")] + [("data", C.c_void_p)]


class nq_page_map(C.Structure):
    _fields_ = [("max_seqs", C.c_int32), ("max_pages", C.c_int32), ("n_pages", C.c_int32), ("page_size", C.c_int32),
                ("table", C.c_void_p), ("held", C.c_void_p), ("ref", C.c_void_p)]


class nq_attn_opts(C.Structure):
    _fields_ = [("scale", C.c_float), ("softcap", C.c_float), ("window", C.c_int32), ("pad", C.c_int32),
                ("slopes", C.c_void_p)]


class nq_tree(C.Structure):
    _fields_ = [("batch", C.c_int32), ("nodes", C.c_int32), ("window", C.c_int32), ("pad", C.c_int32),
                ("parents", C.c_void_p), ("depth", C.c_void_p), ("bits", C.c_void_p)]


def lib():
    """Load libnq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libnq.so is missing at {LIB_PATH}; build it with "
                                   "`python -m quantized_self_speculative_gb300.build` (needs nvcc)")
            L = C.CDLL(LIB_PATH)
            vp, i32, sz, u64, f32 = C.c_void_p, C.c_int, C.c_size_t, C.c_uint64, C.c_float
            W = C.POINTER(nq_weights)
            L.nq_packed_bytes.argtypes = [i32, i32, i32, i32, C.POINTER(sz), C.POINTER(sz), C.POINTER(sz)]
            L.nq_pack_weights.argtypes = [vp, W, vp]
            for name in ("nq_draft_gemv", "nq_verify_gemm"):
                getattr(L, name).argtypes = [W, vp, i32, vp, vp]
            for name in ("nq_draft_gemv_batch", "nq_verify_gemm_batch"):
                getattr(L, name).argtypes = [i32, W, C.POINTER(vp), i32, C.POINTER(vp), vp]
            for name in ("nq_draft_gemv_batch_ws", "nq_verify_gemm_batch_ws"):
                getattr(L, name).argtypes = [i32, W, C.POINTER(vp), i32, C.POINTER(vp), vp, sz, vp]
                getattr(L, name).restype = i32
            L.nq_linear_workspace_bytes.argtypes = [i32, W, i32, i32]
            L.nq_linear_workspace_bytes.restype = sz
            L.spec_accept_workspace_bytes.argtypes = [i32, i32, i32]
            L.spec_accept_workspace_bytes.restype = sz
            L.spec_accept_greedy.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, sz, vp]
            L.spec_accept_sample.argtypes = [vp, vp, vp, i32, i32, i32, f32, vp, u64, vp, vp, vp, sz, vp]
            L.nq_status_string.argtypes = [i32]
            L.nq_status_string.restype = C.c_char_p
            L.nq_get_device_status.argtypes = [vp, C.POINTER(C.c_uint32)]
            L.spec_draft_argmax.argtypes = [vp, i32, i32, vp, i32, vp, sz, vp]
            L.nq_quantize_act_int8.argtypes = [vp, i32, i32, vp, vp, vp]
            L.nq_linear_a8_batch.argtypes = [i32, W, C.POINTER(vp), C.POINTER(vp), i32, i32, C.POINTER(vp), vp]
            for name in ("nq_quantize_act_int8", "nq_linear_a8_batch"):
                getattr(L, name).restype = i32
            KV = C.POINTER(nq_kv_cache)
            L.nq_kv_cache_bytes.argtypes = [i32, i32, i32, i32, i32, C.POINTER(sz), C.POINTER(sz)]
            L.nq_kv_append.argtypes = [KV, vp, vp, i32, vp, vp]
            L.nq_attn_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
            L.nq_attn_workspace_bytes.restype = sz
            L.nq_attn_decode.argtypes = [KV, vp, i32, i32, vp, i32, f32, vp, vp, sz, vp]
            for name in ("nq_kv_cache_bytes", "nq_kv_append", "nq_attn_decode"):
                getattr(L, name).restype = i32
            L.spec_accept_sample_features.argtypes = [vp, vp, vp, i32, i32, i32, f32, vp, u64, vp, vp, vp, vp, sz, vp]
            L.spec_accept_sample_features.restype = i32
            L.nq_embed_rows.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp]
            L.nq_embed_round.argtypes = [vp, i32, i32, vp, vp, i32, i32, vp, vp]
            L.spec_round_commit.argtypes = [vp, vp, i32, i32, vp, vp, i32, vp, vp]
            for name in ("spec_draft_argmax", "nq_embed_rows", "nq_embed_round", "spec_round_commit"):
                getattr(L, name).restype = i32
            i64, RP, PP, PM, AO = C.c_int64, C.POINTER(nq_rope_plan), C.POINTER(nq_page_pool), C.POINTER(nq_page_map), C.POINTER(nq_attn_opts)
            L.nq_rope_rates.argtypes = [i32, C.c_double, i32, C.c_double, i32, vp, C.POINTER(f32)]
            L.nq_rope_mscale.argtypes = [i32, C.c_double, C.POINTER(f32), C.POINTER(f32)]
            L.nq_rope.argtypes = [RP, vp, i32, i64, vp, i32, i32, i32, i32, vp, i32, i64, vp]
            L.nq_page_pool_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32, C.POINTER(sz)]
            L.nq_page_map_init.argtypes = [PM, vp]
            L.nq_page_workspace_bytes.argtypes = [PM, i32]
            L.nq_page_workspace_bytes.restype = sz
            L.nq_page_reserve.argtypes = [PM, PP, vp, vp, vp, i32, vp, vp, sz, vp]
            L.nq_page_fork.argtypes = [PM, vp, vp, vp, i32, vp, sz, vp]
            L.nq_page_truncate.argtypes = [PM, vp, vp, i32, vp]
            L.nq_page_compact.argtypes = [PM, PP, vp, vp, sz, vp]
            L.nq_page_copy.argtypes = [PP, vp, vp, i32, vp]
            L.nq_page_append.argtypes = [PP, i32, PM, RP, vp, vp, vp, i32, i64, vp, vp, i32, i32, vp, vp]
            L.nq_page_read.argtypes = [PP, i32, PM, vp, vp, i32, i32, vp, vp, vp]
            L.nq_page_attn_workspace_bytes.argtypes = [i32, i32, i32, i32]
            L.nq_page_attn_workspace_bytes.restype = sz
            L.nq_page_attn.argtypes = [PP, i32, PM, vp, i64, i32, i32, i32, vp, vp, i32, AO, vp, vp, sz, vp]
            TR = C.POINTER(nq_tree)
            L.nq_tree_plan.argtypes = [TR, vp]
            L.spec_accept_tree.argtypes = [TR, vp, vp, i32, i32, vp, vp, vp, vp]
            L.nq_page_keep.argtypes = [PP, PM, vp, vp, vp, vp, i32, i32, vp]
            L.nq_page_append_at.argtypes = [PP, i32, PM, RP, vp, vp, vp, i32, i64, vp, vp, vp, i32, i32, vp, vp]
            L.nq_rms_norm.argtypes = [vp, i32, i64, vp, i32, i64, vp, i32, f32, i32, i32, vp, i64, vp, vp, vp, vp]
            L.nq_page_attn_tree_workspace_bytes.argtypes = [i32, i32, i32, i32]
            L.nq_page_attn_tree_workspace_bytes.restype = sz
            L.nq_page_attn_tree.argtypes = [PP, i32, PM, vp, i64, i32, vp, vp, i32, AO, TR, vp, vp, sz, vp]
            L.nq_selftest_page_attn_tree.argtypes = [PP, i32, PM, vp, i64, i32, vp, vp, i32, AO, TR, vp, vp, sz, i32, C.c_uint32, vp]
            for name in ("nq_page_attn_tree", "nq_selftest_page_attn_tree", "nq_tree_plan", "spec_accept_tree", "nq_page_keep", "nq_page_append_at", "nq_rms_norm"):
                getattr(L, name).restype = i32
            for name in ("nq_rope_rates", "nq_rope_mscale", "nq_rope", "nq_page_pool_bytes", "nq_page_map_init", "nq_page_reserve",
                         "nq_page_fork", "nq_page_truncate", "nq_page_compact", "nq_page_copy", "nq_page_append",
                         "nq_page_read", "nq_page_attn"):
                getattr(L, name).restype = i32
            L.nq_selftest_bounded_wait.argtypes = [C.c_uint32, vp]
            L.nq_selftest_bounded_wait.restype = i32
            L.nq_selftest_page_attn.argtypes = [PP, i32, PM, vp, i64, i32, i32, i32, vp, vp, i32, AO, vp, vp, sz, i32, C.c_uint32, vp]
            L.nq_selftest_page_attn.restype = i32
            for name in ("nq_packed_bytes", "nq_pack_weights", "nq_draft_gemv", "nq_verify_gemm",
                         "nq_draft_gemv_batch", "nq_verify_gemm_batch", "spec_accept_greedy",
                         "spec_accept_sample", "nq_get_device_status"):
                getattr(L, name).restype = i32
            _lib = L
        return _lib


def status_string(status: int) -> str:
    return lib().nq_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != NQ_OK:
        raise NQError(status, what)


# the current stream's handle without a Stream object around it (3 us less per call), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None or _raw_device is None or not torch.cuda.is_initialized():
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_raw_device())


def _dev(t: torch.Tensor, dtype, what: str) -> int:
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor of {dtype}")
    return t.data_ptr()


# ---------------------------------------------------------------- weights
def packed_bytes(n_out: int, k_in: int, group: int, fmt: int):
    b, r, s = C.c_size_t(), C.c_size_t(), C.c_size_t()
    _check(lib().nq_packed_bytes(n_out, k_in, group, fmt, C.byref(b), C.byref(r), C.byref(s)), "nq_packed_bytes")
    return b.value, r.value, s.value


@dataclass
class PackedLinear:
    """A packed linear layer W [n_out][k_in]; buffers are uint8 device tensors."""
    n_out: int
    k_in: int
    group: int
    fmt: int
    base: torch.Tensor
    resid: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]

    def struct(self) -> nq_weights:
        return nq_weights(self.n_out, self.k_in, self.group, self.fmt, self.base.data_ptr(),
                          None if self.resid is None else self.resid.data_ptr(),
                          None if self.scales is None else self.scales.data_ptr())

    def as_int4(self) -> "PackedLinear":
        """The INT4 view of a NESTED44 layer (same base plane and scales)."""
        return PackedLinear(self.n_out, self.k_in, self.group, FMT_INT4, self.base, None, self.scales)

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.base, self.resid, self.scales) if t is not None)


def alloc_packed(n_out: int, k_in: int, group: int, fmt: int, device=None) -> PackedLinear:
    device = device or torch.device("cuda")
    b, r, s = packed_bytes(n_out, k_in, group, fmt)
    mk = lambda n: torch.empty(n, dtype=torch.uint8, device=device) if n else None
    return PackedLinear(n_out, k_in, group, fmt, mk(b), mk(r), mk(s))


def pack_weights(w: torch.Tensor, fmt: int = FMT_NESTED44, group: int = 128, stream=None) -> PackedLinear:
    n, k = w.shape
    out = alloc_packed(n, k, group, fmt, w.device)
    st = out.struct()
    _check(lib().nq_pack_weights(_dev(w, torch.float32, "w"), C.byref(st), _stream(stream)), "nq_pack_weights")
    return out


def pack_from_host(base, resid, scales, n_out, k_in, group, fmt, device=None) -> PackedLinear:
    """Upload already-packed planes (numpy arrays) to the device."""
    device = device or torch.device("cuda")
    t = lambda a: None if a is None else torch.from_numpy(a.reshape(-1).view("uint8").copy()).to(device)
    return PackedLinear(n_out, k_in, group, fmt, t(base), t(resid), t(scales))


# ---------------------------------------------------------------- linears
def _linear(fn: str, w: PackedLinear, x: torch.Tensor, y: Optional[torch.Tensor], stream) -> torch.Tensor:
    M = x.shape[0]
    if x.shape[-1] != w.k_in:
        raise ValueError("x must be [M][k_in]")
    if y is None:
        y = torch.empty((M, w.n_out), dtype=torch.float32, device=x.device)
    st = w.struct()
    xp = _dev(x, torch.bfloat16, "x") if x.dtype == torch.bfloat16 else _dev(x, torch.int16, "x")
    _check(getattr(lib(), fn)(C.byref(st), xp, M, _dev(y, torch.float32, "y"), _stream(stream)), fn)
    return y


def draft_gemv(w: PackedLinear, x: torch.Tensor, y=None, stream=None) -> torch.Tensor:
    """Draft pass: base plane only.  x: bf16 [M][k_in] -> y fp32 [M][n_out]."""
    return _linear("nq_draft_gemv", w, x, y, stream)


def verify_gemm(w: PackedLinear, x: torch.Tensor, y=None, stream=None) -> torch.Tensor:
    """Verify pass: both planes (8-bit target), or the FP8 / FP16 tiers."""
    return _linear("nq_verify_gemm", w, x, y, stream)


def linear_workspace_bytes(verify: bool, layers: Sequence[PackedLinear], M: int) -> int:
    """Workspace of nq_{draft_gemv,verify_gemm}_batch_ws (0: the tensor-core
    path is not taken for these layers and M)."""
    w = (nq_weights * len(layers))(*[L.struct() for L in layers])
    return lib().nq_linear_workspace_bytes(len(layers), w, M, int(verify))


class LinearBatch:
    """Prebuilt argument arrays for nq_{draft_gemv,verify_gemm}_batch: one
    persistent launch over many independent linears at the same M.  With
    tensor_cores=True the *_batch_ws entry point is used with a workspace
    allocated here (the tensor-memory kernel for M >= 16)."""

    def __init__(self, verify: bool, layers: Sequence[PackedLinear], xs: Sequence[torch.Tensor],
                 ys: Sequence[torch.Tensor], tensor_cores: bool = False):
        n = len(layers)
        assert n == len(xs) == len(ys) and n > 0
        self.fn = "nq_verify_gemm_batch" if verify else "nq_draft_gemv_batch"
        self.M = xs[0].shape[0]
        for L, x, y in zip(layers, xs, ys):
            assert x.shape == (self.M, L.k_in) and y.shape == (self.M, L.n_out)
            _dev(x, torch.bfloat16, "x")
            _dev(y, torch.float32, "y")
        self.count = n
        self.w = (nq_weights * n)(*[L.struct() for L in layers])
        self.x = (C.c_void_p * n)(*[x.data_ptr() for x in xs])
        self.y = (C.c_void_p * n)(*[y.data_ptr() for y in ys])
        self.ws = None
        if tensor_cores:
            self.fn += "_ws"
            nb = lib().nq_linear_workspace_bytes(n, self.w, self.M, int(verify))
            self.ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=xs[0].device)
        self._keep = (list(layers), list(xs), list(ys))

    def __call__(self, stream=None):
        if self.ws is None:
            _check(getattr(lib(), self.fn)(self.count, self.w, self.x, self.M, self.y, _stream(stream)), self.fn)
        else:
            _check(getattr(lib(), self.fn)(self.count, self.w, self.x, self.M, self.y, self.ws.data_ptr(),
                                           self.ws.numel(), _stream(stream)), self.fn)


# ---------------------------------------------------------------- acceptance
def workspace_bytes(B: int, k: int, V: int) -> int:
    return lib().spec_accept_workspace_bytes(B, k, V)


def accept_workspace(B: int, k: int, V: int, device=None) -> torch.Tensor:
    """Zero-filled workspace (the calls leave it ready for reuse)."""
    n = workspace_bytes(B, k, V)
    if n == 0:
        raise NQError(NQ_ERR_ARG, "spec_accept_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def accept_greedy(draft: torch.Tensor, tgt_logits: torch.Tensor, ws: Optional[torch.Tensor] = None,
                  out_tok=None, out_cnt=None, stream=None):
    B, k = draft.shape
    V = tgt_logits.shape[-1]
    if tgt_logits.shape != (B, k + 1, V):
        raise ValueError("tgt_logits must be [B][k+1][V]")
    ws = ws if ws is not None else accept_workspace(B, k, V, draft.device)
    out_tok = out_tok if out_tok is not None else torch.empty((B, k + 1), dtype=torch.int32, device=draft.device)
    out_cnt = out_cnt if out_cnt is not None else torch.empty(B, dtype=torch.int32, device=draft.device)
    _check(lib().spec_accept_greedy(_dev(draft, torch.int32, "draft"), _dev(tgt_logits, torch.float32, "tgt_logits"),
                                    B, k, V, _dev(out_tok, torch.int32, "out_tok"), _dev(out_cnt, torch.int32, "out_cnt"),
                                    _dev(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)), "spec_accept_greedy")
    return out_tok, out_cnt


def accept_sample(draft: torch.Tensor, draft_logits: torch.Tensor, tgt_logits: torch.Tensor, temperature: float,
                  seeds: torch.Tensor, round_: int, ws: Optional[torch.Tensor] = None, out_tok=None, out_cnt=None,
                  stream=None):
    B, k = draft.shape
    V = tgt_logits.shape[-1]
    if tgt_logits.shape != (B, k + 1, V) or draft_logits.shape != (B, k, V):
        raise ValueError("draft_logits must be [B][k][V] and tgt_logits [B][k+1][V]")
    ws = ws if ws is not None else accept_workspace(B, k, V, draft.device)
    out_tok = out_tok if out_tok is not None else torch.empty((B, k + 1), dtype=torch.int32, device=draft.device)
    out_cnt = out_cnt if out_cnt is not None else torch.empty(B, dtype=torch.int32, device=draft.device)
    seeds_p = _dev(seeds, torch.int64, "seeds") if seeds.dtype == torch.int64 else _dev(seeds, torch.uint64, "seeds")
    _check(lib().spec_accept_sample(_dev(draft, torch.int32, "draft"), _dev(draft_logits, torch.float32, "draft_logits"),
                                    _dev(tgt_logits, torch.float32, "tgt_logits"), B, k, V, float(temperature),
                                    seeds_p, int(round_) & (2**64 - 1), _dev(out_tok, torch.int32, "out_tok"),
                                    _dev(out_cnt, torch.int32, "out_cnt"), _dev(ws, torch.uint8, "ws"), ws.numel(),
                                    _stream(stream)), "spec_accept_sample")
    return out_tok, out_cnt


# ---------------------------------------------------------------- round bookkeeping
def draft_argmax(logits: torch.Tensor, tok: torch.Tensor, tok_stride: int = 1, ws: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """tok[m * tok_stride] = argmax of logits row m (fp32 [M][V]); tok is an
    int32 tensor viewed flat (it may be a strided slice's base)."""
    M, V = logits.shape
    ws = ws if ws is not None else accept_workspace(M, 0, V, logits.device)
    _check(lib().spec_draft_argmax(_dev(logits, torch.float32, "logits"), M, V, tok.data_ptr(), int(tok_stride),
                                   _dev(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)), "spec_draft_argmax")
    return tok


def embed_rows(table: torch.Tensor, ids: torch.Tensor, M: int, ids_stride: int = 1, out=None, stream=None):
    """out[m] = table[ids[m * ids_stride]] (table bf16 [V][d]); ids int32."""
    V, d = table.shape
    out = out if out is not None else torch.empty((M, d), dtype=torch.bfloat16, device=table.device)
    _check(lib().nq_embed_rows(_dev(table, torch.bfloat16, "table"), V, d, ids.data_ptr(), int(ids_stride), M,
                               _dev(out, torch.bfloat16, "out"), _stream(stream)), "nq_embed_rows")
    return out


def embed_round(table: torch.Tensor, x0: torch.Tensor, draft: Optional[torch.Tensor], B: int, k: int, out=None,
                stream=None):
    """The verify rows of a round: out[b][0] = table[x0[b]], out[b][j] = table[draft[b][j-1]]."""
    V, d = table.shape
    out = out if out is not None else torch.empty((B * (k + 1), d), dtype=torch.bfloat16, device=table.device)
    _check(lib().nq_embed_round(_dev(table, torch.bfloat16, "table"), V, d, x0.data_ptr(),
                                None if draft is None else draft.data_ptr(), B, k, _dev(out, torch.bfloat16, "out"),
                                _stream(stream)), "nq_embed_round")
    return out


def round_commit(out_tok: torch.Tensor, out_cnt: torch.Tensor, seq: torch.Tensor, seq_len: torch.Tensor,
                 x0: torch.Tensor, stream=None) -> None:
    """Append the emitted tokens to seq [B][max_len] (int32), advance seq_len,
    set x0 to each row's last emitted token (all in place, on the device)."""
    B, k1 = out_tok.shape
    _check(lib().spec_round_commit(_dev(out_tok, torch.int32, "out_tok"), _dev(out_cnt, torch.int32, "out_cnt"), B,
                                   k1 - 1, _dev(seq, torch.int32, "seq"), _dev(seq_len, torch.int32, "seq_len"),
                                   seq.shape[1], _dev(x0, torch.int32, "x0"), _stream(stream)), "spec_round_commit")


def accept_sample_features(draft: torch.Tensor, draft_logits: torch.Tensor, tgt_logits: torch.Tensor,
                           temperature: float, seeds: torch.Tensor, round_: int, ws: Optional[torch.Tensor] = None,
                           out_tok=None, out_cnt=None, features=None, stream=None):
    """spec_accept_sample plus SpecKV's step features per row: (mean entropy,
    mean confidence, max entropy, min confidence) of the k drafted positions."""
    B, k = draft.shape
    V = tgt_logits.shape[-1]
    ws = ws if ws is not None else accept_workspace(B, k, V, draft.device)
    out_tok = out_tok if out_tok is not None else torch.empty((B, k + 1), dtype=torch.int32, device=draft.device)
    out_cnt = out_cnt if out_cnt is not None else torch.empty(B, dtype=torch.int32, device=draft.device)
    features = features if features is not None else torch.empty((B, 4), dtype=torch.float32, device=draft.device)
    seeds_p = _dev(seeds, torch.int64, "seeds") if seeds.dtype == torch.int64 else _dev(seeds, torch.uint64, "seeds")
    _check(lib().spec_accept_sample_features(
        _dev(draft, torch.int32, "draft"), _dev(draft_logits, torch.float32, "draft_logits"),
        _dev(tgt_logits, torch.float32, "tgt_logits"), B, k, V, float(temperature), seeds_p, int(round_) & (2**64 - 1),
        _dev(out_tok, torch.int32, "out_tok"), _dev(out_cnt, torch.int32, "out_cnt"),
        _dev(features, torch.float32, "features"), _dev(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)),
        "spec_accept_sample_features")
    return out_tok, out_cnt, features


# ---------------------------------------------------------------- int8 activations (W4A8 -> W8A8)
def quantize_act_int8(x: torch.Tensor, xq=None, sx=None, stream=None):
    """bf16 [M][K] -> (int8 codes [M][K], fp32 row scales [M])."""
    M, K = x.shape
    xq = xq if xq is not None else torch.empty((M, K), dtype=torch.int8, device=x.device)
    sx = sx if sx is not None else torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib().nq_quantize_act_int8(_dev(x, torch.bfloat16, "x"), M, K, _dev(xq, torch.int8, "xq"),
                                      _dev(sx, torch.float32, "sx"), _stream(stream)), "nq_quantize_act_int8")
    return xq, sx


class LinearA8Batch:
    """Prebuilt argument arrays for nq_linear_a8_batch (one launch over many
    linears at the same M, int8 activation codes and row scales)."""

    def __init__(self, verify: bool, layers: Sequence[PackedLinear], xqs, sxs, ys):
        n = len(layers)
        self.verify, self.count, self.M = int(verify), n, xqs[0].shape[0]
        self.w = (nq_weights * n)(*[L.struct() for L in layers])
        self.xq = (C.c_void_p * n)(*[t.data_ptr() for t in xqs])
        self.sx = (C.c_void_p * n)(*[t.data_ptr() for t in sxs])
        self.y = (C.c_void_p * n)(*[t.data_ptr() for t in ys])
        self._keep = (list(layers), list(xqs), list(sxs), list(ys))

    def __call__(self, stream=None):
        _check(lib().nq_linear_a8_batch(self.count, self.w, self.xq, self.sx, self.M, self.verify, self.y,
                                        _stream(stream)), "nq_linear_a8_batch")


def linear_a8(w: PackedLinear, xq: torch.Tensor, sx: torch.Tensor, verify: bool, y=None, stream=None):
    """One int8-activation linear: y fp32 [M][n_out]."""
    M = xq.shape[0]
    y = y if y is not None else torch.empty((M, w.n_out), dtype=torch.float32, device=xq.device)
    LinearA8Batch(verify, [w], [xq], [sx], [y])(stream)
    return y


# ---------------------------------------------------------------- nested KV cache
class KVCache:
    """One layer's nested KV cache (device buffers allocated here, uint8;
    BitNest Fig. 4): planes [batch][heads_kv][max_len][head_dim/2], fp16
    scales [batch][heads_kv][max_len][head_dim/group], for K and for V."""

    def __init__(self, batch: int, heads_kv: int, head_dim: int, group: int, max_len: int, device=None):
        device = device or torch.device("cuda")
        pb, sb = C.c_size_t(), C.c_size_t()
        _check(lib().nq_kv_cache_bytes(batch, heads_kv, head_dim, group, max_len, C.byref(pb), C.byref(sb)),
               "nq_kv_cache_bytes")
        self.batch, self.heads_kv, self.head_dim, self.group, self.max_len = batch, heads_kv, head_dim, group, max_len
        mk = lambda n: torch.zeros(n, dtype=torch.uint8, device=device)
        self.k_base, self.k_resid, self.k_scales = mk(pb.value), mk(pb.value), mk(sb.value)
        self.v_base, self.v_resid, self.v_scales = mk(pb.value), mk(pb.value), mk(sb.value)
        self.plane_bytes, self.scale_bytes = pb.value, sb.value

    def struct(self) -> nq_kv_cache:
        return nq_kv_cache(self.batch, self.heads_kv, self.head_dim, self.group, self.max_len, 0,
                           self.k_base.data_ptr(), self.k_resid.data_ptr(), self.k_scales.data_ptr(),
                           self.v_base.data_ptr(), self.v_resid.data_ptr(), self.v_scales.data_ptr())

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, pos: torch.Tensor, stream=None) -> None:
        """Quantise k_new, v_new fp32 [batch][heads_kv][n][head_dim] into rows pos[b] .."""
        n = k_new.shape[2]
        st = self.struct()
        _check(lib().nq_kv_append(C.byref(st), _dev(k_new, torch.float32, "k_new"), _dev(v_new, torch.float32, "v_new"),
                                  n, _dev(pos, torch.int32, "pos"), _stream(stream)), "nq_kv_append")

    def attention(self, q: torch.Tensor, lens: torch.Tensor, planes: int, scale: float, out=None, ws=None,
                  stream=None) -> torch.Tensor:
        """softmax(scale q K^T) V over the 4-bit (planes=1) or 8-bit (planes=2)
        view; q fp32 [batch][M][heads_q][head_dim]."""
        B, M, Hq, d = q.shape
        out = out if out is not None else torch.empty_like(q)
        need = lib().nq_attn_workspace_bytes(B, M, Hq, d, self.max_len)
        ws = ws if ws is not None else torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
        st = self.struct()
        _check(lib().nq_attn_decode(C.byref(st), _dev(q, torch.float32, "q"), M, Hq, _dev(lens, torch.int32, "lens"),
                                    int(planes), float(scale), _dev(out, torch.float32, "out"),
                                    _dev(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)), "nq_attn_decode")
        return out

    def host_dict(self):
        """The cache buffers as numpy arrays shaped for the oracle."""
        sh = (self.batch, self.heads_kv, self.max_len)
        p = lambda t: t.cpu().numpy().reshape(*sh, self.head_dim // 2)
        sc = lambda t: t.cpu().numpy().view("uint16").reshape(*sh, self.head_dim // self.group)
        return dict(k_base=p(self.k_base), k_resid=p(self.k_resid), k_scales=sc(self.k_scales),
                    v_base=p(self.v_base), v_resid=p(self.v_resid), v_scales=sc(self.v_scales))


# ---------------------------------------------------------------- memory of the calls below
def _empty(shape, dtype, device, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """A new tensor that the stream may write at once: its memory comes from that
    stream's share of the allocator, whose earlier users the stream waits for."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _zeros(shape, dtype, device, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """The same, cleared on that stream."""
    if stream is None:
        return torch.zeros(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.zeros(shape, dtype=dtype, device=device)


class _Scratch:
    """Workspaces of the calls on one object, kept from call to call (a fork and a
    reservation take 37 us instead of 43, the host's share being all of it): one
    per stream, whose calls follow each other, and per host thread, as two threads'
    launches may interleave.  A captured call takes memory of its graph, a call
    with a stream argument memory of that stream."""

    def __init__(self, device):
        self.device, self.kept = device, {}

    def get(self, need: int, stream: Optional[torch.cuda.Stream], handle: int) -> torch.Tensor:
        if stream is not None or torch.cuda.is_current_stream_capturing():
            return _empty(need, torch.uint8, self.device, stream)
        key = handle, threading.get_ident()
        ws = self.kept.get(key)
        if ws is None or ws.numel() < need:
            ws = self.kept[key] = torch.empty(need, dtype=torch.uint8, device=self.device)
        return ws


# ---------------------------------------------------------------- rotary positions
_DT = {torch.float32: 0, torch.bfloat16: 1}


def _heads(t: torch.Tensor, T: int, H: int, D: int, dtype, what: str) -> int:
    """Address of the heads of T tokens [T][H][D], each token's contiguous."""
    st = t.stride()
    if not t.is_cuda or t.dtype is not dtype or t.shape != (T, H, D) or st[2] != 1 or (st[1] != D and H > 1):
        raise ValueError(f"{what} must be a CUDA tensor of {dtype}, shape {(T, H, D)}, contiguous within a token")
    return t.data_ptr()


def _token_stride(t: torch.Tensor) -> int:
    T, H, D = t.shape
    return t.stride(0) if T > 1 else H * D


class Rope:
    """The rates of a rotation (nq_rope_rates) on the device.  layout "half" or
    "interleaved"; scaling "none", "linear", "ntk" or "parts"."""

    def __init__(self, rot_dim: int, theta: float = 10000.0, layout: str = "half", scaling: str = "none",
                 factor: float = 1.0, old_len: int = 0, device=None):
        rates = torch.empty(max(rot_dim // 2, 1), dtype=torch.int64)
        ms, lo = C.c_float(), C.c_float()
        layouts, kinds = ("half", "interleaved"), ("none", "linear", "ntk", "parts")
        if layout not in layouts or scaling not in kinds:
            raise ValueError(f"layout is one of {layouts}, scaling one of {kinds}")
        _check(lib().nq_rope_rates(rot_dim, float(theta), kinds.index(scaling), float(factor), int(old_len),
                                   rates.data_ptr(), C.byref(ms)), "nq_rope_rates")
        _check(lib().nq_rope_mscale(kinds.index(scaling), float(factor), C.byref(ms), C.byref(lo)), "nq_rope_mscale")
        self.rot_dim, self.mscale = rot_dim, ms.value
        self.rates = rates.to(device or torch.device("cuda"))
        self.struct = nq_rope_plan(rot_dim, layouts.index(layout), ms.value, lo.value, self.rates.data_ptr())
        self.ref = C.byref(self.struct)


def rope(x: torch.Tensor, pos: torch.Tensor, plan: Rope, out: Optional[torch.Tensor] = None, inverse: bool = False,
         out_dtype=None, stream=None) -> torch.Tensor:
    """Rotate x [T][heads][head_dim] (fp32 or bf16; tokens may be strided) by pos
    int32 [T]; out defaults to a new contiguous tensor of out_dtype (x's).
    inverse turns back: the gradient of the rotation."""
    if x.dim() != 3 or x.dtype not in _DT:
        raise ValueError("x must be fp32 or bf16 [T][heads][head_dim]")
    T, H, D = x.shape
    if out is None:
        out = _empty((T, H, D), out_dtype or x.dtype, x.device, stream)
    elif out.dtype not in _DT or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out must be fp32 or bf16, of out_dtype")
    if pos.shape != (T,):
        raise ValueError("pos must be int32 [T]")
    if T == 0:
        return out
    _check(lib().nq_rope(plan.ref, _heads(x, T, H, D, x.dtype, "x"), _DT[x.dtype], _token_stride(x),
                         _dev(pos, torch.int32, "pos"), T, H, D, int(inverse), _heads(out, T, H, D, out.dtype, "out"),
                         _DT[out.dtype], _token_stride(out), _stream(stream)), "nq_rope")
    return out


# ---------------------------------------------------------------- between two linears
def _matrix(t: torch.Tensor, M: int, K: int, what: str):
    """Address, type and row stride of fp32 or bf16 [M][K], each row contiguous."""
    kind = _DT.get(t.dtype)
    if kind is None or not t.is_cuda or t.shape != (M, K) or not (t.is_contiguous() or t.stride(1) == 1 or K == 1):
        raise ValueError(f"{what} must be a CUDA tensor of fp32 or bf16, shape {(M, K)}, contiguous within a row")
    return t.data_ptr(), kind, t.stride(0) if M > 1 else K


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, add: Optional[torch.Tensor] = None,
             quantize: bool = False, sum_out: Optional[torch.Tensor] = None, y=None, xq=None, sx=None, stream=None):
    """Root-mean-square norm of the rows of x [M][K] (fp32 or bf16; rows may be
    strided), of x + add where add is given (nq_rms_norm).  Returns (s, y): s the
    sum in x's type (in sum_out, which may be x; x itself without add), y bf16; with
    quantize (s, xq, sx): int8 codes and fp32 row scales for LinearA8Batch."""
    if x.dim() != 2:
        raise ValueError("x must be fp32 or bf16 [M][K]")
    M, K = shape = x.shape
    xp, xt, xs = _matrix(x, M, K, "x")
    wp, wt = None, 0
    if weight is not None:
        wt = _DT.get(weight.dtype)
        if wt is None or weight.shape != (K,) or not weight.is_cuda or not weight.is_contiguous():
            raise ValueError("weight must be a contiguous CUDA tensor of fp32 or bf16 [K]")
        wp = weight.data_ptr()
    if (y is not None) if quantize else (xq is not None or sx is not None):
        raise ValueError("y without quantize, xq and sx with it")
    if add is None:
        if sum_out is not None:
            raise ValueError("sum_out comes with add and has x's type")
        s, ap, at, as_, sp, ss = x, None, 0, 0, None, 0
    else:
        ap, at, as_ = _matrix(add, M, K, "add")
        s = sum_out if sum_out is not None else _empty(shape, x.dtype, x.device, stream)
        if s.dtype != x.dtype:
            raise ValueError("sum_out comes with add and has x's type")
        sp, _, ss = _matrix(s, M, K, "sum_out")
    if quantize:
        xq = xq if xq is not None else _empty(shape, torch.int8, x.device, stream)
        sx = sx if sx is not None else _empty((M,), torch.float32, x.device, stream)
        if xq.shape != shape or sx.shape != (M,):
            raise ValueError("xq must be int8 [M][K], sx fp32 [M]")
        out = None, _dev(xq, torch.int8, "xq"), _dev(sx, torch.float32, "sx")
    else:
        y = y if y is not None else _empty(shape, torch.bfloat16, x.device, stream)
        if y.shape != shape:
            raise ValueError("y must be bf16 [M][K]")
        out = _dev(y, torch.bfloat16, "y"), None, None
    if M:
        _check(lib().nq_rms_norm(xp, xt, xs, ap, at, as_, wp, wt, eps, M, K, sp, ss, *out, _stream(stream)), "nq_rms_norm")
    return (s, xq, sx) if quantize else (s, y)


# ---------------------------------------------------------------- trees of drafted tokens
class Tree:
    """Trees of drafted tokens, one per sequence (nq_tree): parents int32
    [batch][nodes], each below its node's number; -1 follows the committed rows, less
    marks a node that is not used.  By convention node 0 is the last committed
    token.  Made once a round: depth int32 [batch][nodes] (-1: not used) and bits
    int32 [batch][nodes][ceil(nodes / 32)] serve all layers.  window as in the
    attention that uses it."""

    def __init__(self, parents: torch.Tensor, window: int = 0, stream=None):
        if parents.dim() != 2:
            raise ValueError("parents must be int32 [batch][nodes]")
        self.batch, self.nodes = parents.shape
        self.parents, self.window = parents, int(window)
        p = _dev(parents, torch.int32, "parents")
        self.depth = _empty((self.batch, self.nodes), torch.int32, parents.device, stream)
        self.bits = _empty((self.batch, self.nodes, -(-self.nodes // 32)), torch.int32, parents.device, stream)
        self.struct = nq_tree(self.batch, self.nodes, self.window, 0, p, self.depth.data_ptr(), self.bits.data_ptr())
        self.ref = C.byref(self.struct)
        if self.batch:
            _check(lib().nq_tree_plan(self.ref, _stream(stream)), "nq_tree_plan")

    def positions(self, base: torch.Tensor, stream=None) -> torch.Tensor:
        """Positions int32 [batch][nodes] of the nodes above base int32 [batch] committed rows (a node not used: base's).
        stream: the plan's, where that was made on one."""
        if stream is None:
            return base[:, None] + self.depth.clamp(min=0)
        with torch.cuda.stream(stream):
            return base[:, None] + self.depth.clamp(min=0)


def accept_tree(tokens: torch.Tensor, logits: torch.Tensor, tree: Tree, width: Optional[int] = None, out_tok=None, out_cnt=None,
                path=None, stream=None):
    """Greedy acceptance along the trees (spec_accept_tree): tokens int32
    [batch][nodes], logits fp32 [batch][nodes][V].  Returns the emitted tokens
    [batch][width], their number [batch] and the nodes that emitted them [batch][width]."""
    B, M = tree.batch, tree.nodes
    width = M if width is None else int(width)
    if tokens.shape != (B, M) or logits.dim() != 3 or logits.shape[:2] != (B, M):
        raise ValueError("tokens must be [batch][nodes] and logits [batch][nodes][V]")
    mk = lambda t, *s: t if t is not None else _empty(s, torch.int32, logits.device, stream)  # noqa: E731
    out_tok, out_cnt, path = mk(out_tok, B, width), mk(out_cnt, B), mk(path, B, width)
    if out_tok.shape != (B, width) or out_cnt.shape != (B,) or path.shape != (B, width):
        raise ValueError("out_tok and path must be int32 [batch][width], out_cnt int32 [batch]")
    if B:
        _check(lib().spec_accept_tree(tree.ref, _dev(tokens, torch.int32, "tokens"), _dev(logits, torch.float32, "logits"),
                                      logits.shape[2], width, _dev(out_tok, torch.int32, "out_tok"),
                                      _dev(out_cnt, torch.int32, "out_cnt"), _dev(path, torch.int32, "path"), _stream(stream)),
               "spec_accept_tree")
    return out_tok, out_cnt, path


# ---------------------------------------------------------------- paged KV cache
class PageMap:
    """Which pages the sequence slots hold (nq_page_map).  Device tensors int32:
    table [max_seqs][max_pages], held [max_seqs], ref [n_pages]; those not given
    are made and cleared.  A given table alone makes a map to append to and
    read, whose pages the caller keeps."""

    def __init__(self, max_seqs: int, max_pages: int, n_pages: int, page_size: int, table=None, held=None, ref=None,
                 device=None, stream=None):
        dev = table.device if table is not None else device or torch.device("cuda")
        mk = lambda *s: _empty(s, torch.int32, dev, stream)  # noqa: E731
        fresh = table is None
        if fresh and (held is not None or ref is not None):
            raise ValueError("held and ref come with a table")
        if fresh:
            table, held, ref = mk(max_seqs, max_pages), mk(max_seqs), mk(n_pages)
        if (held is None) != (ref is None):
            raise ValueError("held and ref come together")
        for t, shape in ((table, (max_seqs, max_pages)), (held, (max_seqs,)), (ref, (n_pages,))):
            if t is not None and tuple(t.shape) != shape:
                raise ValueError(f"table, held and ref must have shapes {(max_seqs, max_pages)}, {(max_seqs,)}, {(n_pages,)}")
        self.table, self.held, self.ref = table, held, ref
        self.max_seqs, self.max_pages, self.n_pages, self.page_size = max_seqs, max_pages, n_pages, page_size
        p = lambda t, what: None if t is None else _dev(t, torch.int32, what)  # noqa: E731
        self.struct = nq_page_map(max_seqs, max_pages, n_pages, page_size, p(table, "table"), p(held, "held"), p(ref, "ref"))
        self.ptr = C.byref(self.struct)
        self._ws_bytes = {}              # workspace size by the number of sequences
        self._scratch = _Scratch(dev)
        if fresh:
            _check(lib().nq_page_map_init(self.ptr, _stream(stream)), "nq_page_map_init")

    def _work(self, n: int, ws: Optional[torch.Tensor], stream, handle: int) -> torch.Tensor:
        """The given workspace, or one for n sequences."""
        if ws is not None:
            _dev(ws, torch.uint8, "ws")
            return ws
        need = self._ws_bytes.get(n)
        if need is None:
            need = self._ws_bytes[n] = max(lib().nq_page_workspace_bytes(self.ptr, n), 16)
        return self._scratch.get(need, stream, handle)

    @staticmethod
    def _list(t: torch.Tensor, n: int, what: str) -> int:
        if t.shape != (n,):
            raise ValueError(f"{what} must be int32 [{n}]")
        return _dev(t, torch.int32, what)

    def reserve(self, pool: Optional["PagePool"], seqs, first, last, granted=None, ws=None, stream=None) -> torch.Tensor:
        """Pages for rows first[i] .. last[i]-1 of slots seqs[i], shared ones
        copied first; returns int32 [n], 1 where served."""
        n = seqs.shape[0]
        lists = self._list(seqs, n, "seqs"), self._list(first, n, "first"), self._list(last, n, "last")
        on = _stream(stream)
        granted = granted if granted is not None else _empty(n, torch.int32, seqs.device, stream)
        if n == 0:
            return granted
        ws = self._work(n, ws, stream, on)
        _check(lib().nq_page_reserve(self.ptr, None if pool is None else pool.ptr, *lists, n,
                                     self._list(granted, n, "granted"), ws.data_ptr(), ws.numel(), on),
               "nq_page_reserve")
        return granted

    def fork(self, src, dst, rows, ws=None, stream=None) -> None:
        """Slot dst[i] shares slot src[i]'s first rows[i] rows (all pairs at once)."""
        n = src.shape[0]
        lists = self._list(src, n, "src"), self._list(dst, n, "dst"), self._list(rows, n, "rows")
        if n == 0:
            return
        on = _stream(stream)
        ws = self._work(n, ws, stream, on)
        _check(lib().nq_page_fork(self.ptr, *lists, n, ws.data_ptr(), ws.numel(), on), "nq_page_fork")

    def truncate(self, seqs, rows, stream=None) -> None:
        """Slot seqs[i] keeps the pages of its first rows[i] rows."""
        n = seqs.shape[0]
        lists = self._list(seqs, n, "seqs"), self._list(rows, n, "rows")
        if n == 0:
            return
        _check(lib().nq_page_truncate(self.ptr, *lists, n, _stream(stream)), "nq_page_truncate")

    def compact(self, pool: "PagePool", used=None, ws=None, stream=None) -> torch.Tensor:
        """Move the pages in use to the lowest ids; returns how many (int32 [1])."""
        on = _stream(stream)
        used = used if used is not None else _empty(1, torch.int32, self.table.device, stream)
        ws = self._work(1, ws, stream, on)
        _check(lib().nq_page_compact(self.ptr, pool.ptr, self._list(used, 1, "used"), ws.data_ptr(), ws.numel(), on),
               "nq_page_compact")
        return used


class PagePool:
    """The pages of all layers (nq_page_pool); data uint8, made and cleared here
    (on `stream`) unless given."""

    def __init__(self, layers: int, n_pages: int, page_size: int, heads_kv: int, head_dim: int, fmt: int = KV_NESTED44,
                 group: int = 128, data: Optional[torch.Tensor] = None, device=None, stream=None):
        n = C.c_size_t()
        _check(lib().nq_page_pool_bytes(layers, n_pages, page_size, heads_kv, head_dim, group, fmt, C.byref(n)),
               "nq_page_pool_bytes")
        self.bytes = n.value
        if data is None:
            data = _zeros(n.value, torch.uint8, device or torch.device("cuda"), stream)
        if data.numel() != n.value:
            raise ValueError(f"data must hold {n.value} bytes")
        self.data, self.layers, self.n_pages, self.page_size = data, layers, n_pages, page_size
        self.heads_kv, self.head_dim, self.group, self.fmt = heads_kv, head_dim, group, fmt
        self.struct = nq_page_pool(layers, n_pages, page_size, heads_kv, head_dim, group, fmt, 0,
                                   _dev(data, torch.uint8, "data"))
        self.ptr = C.byref(self.struct)
        self._attn_bytes = {}            # workspace size by (M, heads_q), with and without a tree
        self._scratch = _Scratch(data.device)

    def copy_pages(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Copy pages src[i] to dst[i] in every layer."""
        n = src.shape[0]
        lists = PageMap._list(src, n, "src"), PageMap._list(dst, n, "dst")
        if n == 0:
            return
        _check(lib().nq_page_copy(self.ptr, *lists, n, _stream(stream)), "nq_page_copy")

    def append(self, layer: int, pmap: PageMap, k: torch.Tensor, v: torch.Tensor, seqs: torch.Tensor, pos: torch.Tensor,
               rope: Optional[Rope] = None, q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
               stream=None, at: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
        """Store k, v [T][heads_kv][head_dim] (fp32 or bf16) as row pos[t] of slot
        seqs[t], k rotated by pos (by at, where given: a tree's nodes); with q
        [T][heads_q][head_dim] returns the rotated queries in bf16.  q, k and v may
        be columns of one tensor."""
        T, H, D = k.shape[0], self.heads_kv, self.head_dim
        if k.dtype not in _DT:
            raise ValueError("k must be fp32 or bf16")
        stride = _token_stride(k)
        Hq = 0 if q is None else q.shape[1]
        if T > 1 and (v.stride(0) != stride or (q is not None and q.stride(0) != stride)):
            raise ValueError("q, k and v must have one stride between tokens")
        if T == 1:
            stride = max(H, Hq) * D
        if q is not None and q_out is None:
            q_out = _empty((T, Hq, D), torch.bfloat16, q.device, stream)
        if T == 0:
            return q_out
        rows = PageMap._list(pos, T, "pos")
        _check(lib().nq_page_append_at(self.ptr, layer, pmap.ptr, None if rope is None else rope.ref,
                                       None if q is None else _heads(q, T, Hq, D, k.dtype, "q"),
                                       _heads(k, T, H, D, k.dtype, "k"), _heads(v, T, H, D, k.dtype, "v"), _DT[k.dtype],
                                       stride, PageMap._list(seqs, T, "seqs"), rows,
                                       rows if at is None else PageMap._list(at, T, "at"), T, Hq,
                                       None if q is None else self._rows(q_out, (T, Hq, D), "q_out"), _stream(stream)),
               "nq_page_append_at")
        return q_out

    def keep(self, pmap: PageMap, seqs: torch.Tensor, first: torch.Tensor, path: torch.Tensor, count: torch.Tensor,
             stream=None) -> None:
        """Rows first[i] + path[i][j] of slot seqs[i] become rows first[i] + j,
        j < count[i], in every layer: the accepted path (int32 [n][width], rising) of
        a tree whose nodes were appended from row first[i] on."""
        if path.dim() != 2:
            raise ValueError("path must be int32 [n][width]")
        n, width = path.shape
        lists = (PageMap._list(seqs, n, "seqs"), PageMap._list(first, n, "first"), _dev(path, torch.int32, "path"),
                 PageMap._list(count, n, "count"))
        if n == 0 or width == 0:
            return
        _check(lib().nq_page_keep(self.ptr, pmap.ptr, *lists, n, width, _stream(stream)), "nq_page_keep")

    @staticmethod
    def _rows(t: torch.Tensor, shape, what: str) -> int:
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{what} must have shape {tuple(shape)}")
        return _dev(t, torch.bfloat16, what)

    def read(self, layer: int, pmap: PageMap, seqs: torch.Tensor, pos: torch.Tensor, planes: int = 2, k_out=None,
             v_out=None, stream=None):
        """The stored K and V rows pos[t] of slots seqs[t] as bf16 [T][heads_kv][head_dim]."""
        T = seqs.shape[0]
        shape = (T, self.heads_kv, self.head_dim)
        mk = lambda t: t if t is not None else _empty(shape, torch.bfloat16, seqs.device, stream)  # noqa: E731
        k_out, v_out = mk(k_out), mk(v_out)
        if T:
            _check(lib().nq_page_read(self.ptr, layer, pmap.ptr, PageMap._list(seqs, T, "seqs"),
                                      PageMap._list(pos, T, "pos"), T, int(planes), self._rows(k_out, shape, "k_out"),
                                      self._rows(v_out, shape, "v_out"), _stream(stream)), "nq_page_read")
        return k_out, v_out

    @staticmethod
    def _queries(q: torch.Tensor):
        """Address of q [batch][M][heads][head_dim] and the elements between its batch * M rows."""
        B, M, H, D = q.shape
        if q.is_contiguous():
            return _dev(q, torch.bfloat16, "q"), H * D
        st = q.stride()
        step = st[1] if M > 1 else st[0] if B > 1 else H * D
        if (not q.is_cuda or q.dtype != torch.bfloat16 or st[3] != 1 or (st[2] != D and H > 1)
                or (B > 1 and M > 1 and st[0] != M * st[1])):
            raise ValueError("q must be a CUDA tensor of torch.bfloat16, its batch * M rows evenly spaced and each contiguous")
        return q.data_ptr(), step

    def attention(self, layer: int, pmap: PageMap, q: torch.Tensor, lens: torch.Tensor, planes: int, scale: float,
                  seqs: Optional[torch.Tensor] = None, softcap: float = 0.0, window: int = 0,
                  slopes: Optional[torch.Tensor] = None, out=None, ws=None, stream=None,
                  tree: Optional[Tree] = None) -> torch.Tensor:
        """Attention of the last M rows of each sequence, q bf16 [batch][M][heads_q]
        [head_dim] (its batch * M rows may be strided, each contiguous); sequence
        b is slot seqs[b] (slot b without seqs) of lens[b] rows.  softcap, window and slopes (fp32 [heads_q]) as in nq_attn_opts.
        With a tree (of the same window) the M rows are its nodes: each sees the rows
        before them, the nodes above it and itself (nq_page_attn_tree)."""
        B, M, Hq, D = q.shape
        if D != self.head_dim:
            raise ValueError("q must have the pool's head_dim")
        if slopes is not None and slopes.shape != (Hq,):
            raise ValueError("slopes must be fp32 [heads_q]")
        given = (*self._queries(q), B, M, Hq, None if seqs is None else PageMap._list(seqs, B, "seqs"),
                 PageMap._list(lens, B, "lens"), int(planes))
        if tree is not None and (tree.batch, tree.nodes) != (B, M):
            raise ValueError("q must have the tree's batch and nodes")
        on = _stream(stream)
        if out is None:
            out = _empty(q.shape, q.dtype, q.device, stream)
        if B == 0:
            return out
        if ws is None:
            need = self._attn_bytes.get((M, Hq, tree is None))
            if need is None:
                size = lib().nq_page_attn_workspace_bytes if tree is None else lib().nq_page_attn_tree_workspace_bytes
                need = self._attn_bytes[M, Hq, tree is None] = max(size(M, Hq, self.heads_kv, D), 16)
            ws = self._scratch.get(need, stream, on)
        else:
            _dev(ws, torch.uint8, "ws")
        o = nq_attn_opts(float(scale), float(softcap), int(window), 0,
                         None if slopes is None else _dev(slopes, torch.float32, "slopes"))
        if tree is not None:
            _check(lib().nq_page_attn_tree(self.ptr, layer, pmap.ptr, given[0], given[1], *given[4:], C.byref(o), tree.ref,
                                           self._rows(out, (B, M, Hq, D), "out"), ws.data_ptr(), ws.numel(), on), "nq_page_attn_tree")
            return out
        _check(lib().nq_page_attn(self.ptr, layer, pmap.ptr, *given, C.byref(o), self._rows(out, (B, M, Hq, D), "out"),
                                  ws.data_ptr(), ws.numel(), on), "nq_page_attn")
        return out


def selftest_bounded_wait(limit_us: int, stream=None) -> None:
    """Run the bounded-wait diagnostic (a wait that nothing completes gives up
    after limit_us and sets NQ_DEV_TIMEOUT); read the bit with device_status()."""
    _check(lib().nq_selftest_bounded_wait(int(limit_us), _stream(stream)), "nq_selftest_bounded_wait")


def device_status(stream=None) -> int:
    """Read and clear the sticky device status word (NQ_DEV_* bits)."""
    v = C.c_uint32()
    _check(lib().nq_get_device_status(_stream(stream), C.byref(v)), "nq_get_device_status")
    return v.value
