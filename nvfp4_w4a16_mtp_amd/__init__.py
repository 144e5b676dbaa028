"""NVFP4 W4A16 MTP draft-head hot path on AMD gfx950 (MI355X).

Thin ctypes binding over ``libnvfp4_mtp.so`` (C ABI in include/nvfp4_mtp.h).
It only marshals arguments: every step of every operation runs in the HIP
kernels.  PyTorch supplies device memory and the current stream.  If the
library is not built the calls raise -- there is no fallback.

Operations (same names as the C ABI):
  nvfp4_quantize               bf16 W[n, k] -> NVFP4Weight (codes, scales, global)
  w4a16_gemv                   x[m<=8, k] @ W^T
  w4a16_gemv_grouped           the GEMV for several weights sharing x (q|k|v, gate|up)
  w4a16_gemv_embed             the GEMV over [embedding rows of device ids | x_rest]
  w4a16_gemm_m128              x[m, k] @ W^T for prompt-sized m (bf16 MFMA)
  lmhead_gemv_argmax           argmax over the first V rows of h @ W^T
  lmhead_gemv_argmax_logprob   ... plus the top-1 log-probability
  lmhead_gemv_argmax_masked    ... restricted to a grammar's allowed tokens
  lmhead_gemv_argmax_embed     ... with the draft tokens' embedding rows gathered
  lmhead_gemv_argmax_noalloc   lmhead_gemv_argmax on the library's own static scratch
  lmhead_gemv_argmax_fc        ... then the next draft step's fc over the chosen token's embedding row
  embed_from_argmax            embedding rows of device-resident token ids
  moe_w4a16_gemv               top-k routed NVFP4 expert FFN
  moe_w4a16_gemv_trace         ... one token, with per-workgroup phase timestamps
  moe_layer_w4a16              router + routed experts + gated shared expert
  moe_workspace_status         sticky status of a MoE workspace (host query)
  rope_qk                      rotary positions of q and k rows (rope_frequencies makes the table)
  kv8_append                   k and v rows quantised into a paged 8-bit cache (KV8Cache, KV8Seqs)
  rope_kv8_append              ... with q and k rotated in the same launch
  kv8_read                     the cache's values back in bf16
  kv8_attention                attention over that cache (one token to prompt chunks, window and sinks)
  verify_drafts                which drafted tokens stand, the token after them, the cache lengths left
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4_mtp.so")
_lib = None

NVFP4_OUT_F32 = 0
NVFP4_OUT_BF16 = 1
NVFP4_ARGMAX_BF16_KEYS = 1


class _Weight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("global_", ctypes.c_void_p),
                ("n", ctypes.c_int32), ("k", ctypes.c_int32)]


class _MoeWeights(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("gate_codes", ctypes.c_void_p), ("gate_scales", ctypes.c_void_p), ("gate_global", ctypes.c_void_p),
                ("up_codes", ctypes.c_void_p), ("up_scales", ctypes.c_void_p), ("up_global", ctypes.c_void_p),
                ("down_codes", ctypes.c_void_p), ("down_scales", ctypes.c_void_p), ("down_global", ctypes.c_void_p)]


class _HeadRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("dim", ctypes.c_int32)]


class _Rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("mscale", ctypes.c_float)]


class _KV8Cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _KV8Seqs(ctypes.Structure):
    _fields_ = [("cu_rows", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("rows", ctypes.c_int32), ("max_rows", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("max_kv_len", ctypes.c_int32)]


class NVFP4Error(RuntimeError):
    pass


def lib():
    """The loaded HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise NVFP4Error(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                             "or python nvfp4_w4a16_mtp_amd/build.py")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
        WP = ctypes.POINTER(_Weight)
        EP = ctypes.POINTER(_MoeWeights)
        L.nvfp4_quantize.argtypes = [P, i32, i32, P, P, P, P]
        L.w4a16_gemv.argtypes = [P, i32, WP, P, i32, P]
        L.w4a16_gemv_grouped.argtypes = [P, i32, ctypes.POINTER(WP), ctypes.POINTER(P), i32, i32, P]
        L.w4a16_gemm_m128_workspace_bytes.argtypes = [i32, i32, i32]
        L.w4a16_gemm_m128_workspace_bytes.restype = sz
        L.w4a16_gemm_m128.argtypes = [P, i32, WP, P, i32, P, sz, P]
        L.lmhead_gemv_argmax_workspace_bytes.argtypes = [i32, i32]
        L.lmhead_gemv_argmax_workspace_bytes.restype = sz
        L.lmhead_gemv_argmax.argtypes = [P, i32, WP, i32, P, P, P, sz, u32, P]
        L.lmhead_gemv_argmax_noalloc.argtypes = [P, i32, WP, i32, P, P, u32, P]
        L.lmhead_gemv_argmax_logprob.argtypes = [P, i32, WP, i32, P, P, P, P, sz, u32, P]
        L.lmhead_gemv_argmax_masked.argtypes = [P, i32, WP, i32, P, i32, P, P, P, P, sz, u32, P]
        L.embed_from_argmax.argtypes = [P, i32, P, i32, i32, P, ctypes.c_int64, P, P]
        L.w4a16_gemv_embed.argtypes = [P, P, i32, i32, P, i32, WP, P, i32, P]
        L.lmhead_gemv_argmax_embed.argtypes = [P, i32, WP, i32, P, i32, P, P, P, P, i32, i32, P, ctypes.c_int64, P,
                                               P, sz, u32, P]
        L.lmhead_gemv_argmax_fc.argtypes = [P, i32, WP, i32, P, P, P, sz, u32, P, i32, i32, P, WP, P, i32, P]
        L.moe_w4a16_gemv_workspace_bytes.argtypes = [i32, i32, EP]
        L.moe_w4a16_gemv_workspace_bytes.restype = sz
        L.moe_w4a16_gemv.argtypes = [P, i32, P, i32, EP, P, P, P, P, sz, P]
        L.moe_w4a16_gemv_trace_words.argtypes = [i32, i32, EP]
        L.moe_w4a16_gemv_trace_words.restype = sz
        L.moe_w4a16_gemv_trace.argtypes = [P, i32, P, i32, EP, P, P, P, P, sz, P, sz, P]
        L.moe_layer_w4a16_workspace_bytes.argtypes = [i32, i32, EP]
        L.moe_layer_w4a16_workspace_bytes.restype = sz
        L.moe_layer_w4a16.argtypes = [P, i32, WP, i32, EP, WP, WP, WP, P, P, P, P, P, P, sz, P]
        L.moe_workspace_status.argtypes = [P, sz, ctypes.POINTER(u32), P]
        HP, RP, CP, SP = (ctypes.POINTER(t) for t in (_HeadRows, _Rope, _KV8Cache, _KV8Seqs))
        i64, f32 = ctypes.c_int64, ctypes.c_float
        L.rope_qk.argtypes = [HP, HP, HP, HP, i32, P, RP, P]
        L.kv8_append.argtypes = [CP, SP, HP, HP, P]
        L.rope_kv8_append.argtypes = [CP, SP, RP, HP, HP, HP, HP, P]
        L.kv8_read.argtypes = [CP, SP, HP, HP, P]
        L.kv8_attention_workspace_bytes.argtypes = [CP, SP, i32]
        L.kv8_attention_workspace_bytes.restype = sz
        L.kv8_attention.argtypes = [HP, CP, SP, f32, i32, i32, P, i64, P, sz, P]
        L.verify_drafts_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.verify_drafts_workspace_bytes.restype = sz
        L.verify_drafts.argtypes = [P, i32, i64, i32, P, i64, P, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, sz, P]
        L.nvfp4_mtp_last_error.restype = ctypes.c_char_p
        for f in ("nvfp4_quantize", "w4a16_gemv", "w4a16_gemv_grouped", "w4a16_gemm_m128", "lmhead_gemv_argmax",
                  "lmhead_gemv_argmax_noalloc",
                  "lmhead_gemv_argmax_logprob", "lmhead_gemv_argmax_masked", "embed_from_argmax", "lmhead_gemv_argmax_embed",
                  "lmhead_gemv_argmax_fc",
                  "w4a16_gemv_embed",
                  "moe_w4a16_gemv", "moe_w4a16_gemv_trace", "moe_layer_w4a16", "moe_workspace_status",
                  "rope_qk", "kv8_append", "rope_kv8_append", "kv8_read", "kv8_attention", "verify_drafts"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = lib().nvfp4_mtp_last_error().decode(errors="replace")
        raise NVFP4Error(f"{what} failed ({rc}): {msg}")


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _as_bf16(t: torch.Tensor) -> torch.Tensor:
    if t.dtype == torch.bfloat16:
        return t
    if t.dtype in (torch.int16, torch.uint16):
        return t.view(torch.bfloat16)
    raise TypeError(f"expected bf16 (or 16-bit bit patterns), got {t.dtype}")


def _dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


@dataclass
class NVFP4Weight:
    """One NVFP4 matrix W[n, k] on the device: codes [n, k/2] u8, scales
    [n, k/16] u8 (E4M3FN), glob 4 x fp32 = the 16-byte nvfp4_global struct
    {dec, enc, amax, flags}."""
    codes: torch.Tensor
    scales: torch.Tensor
    glob: torch.Tensor
    n: int
    k: int

    def desc(self) -> _Weight:
        return _Weight(self.codes.data_ptr(), self.scales.data_ptr(), self.glob.data_ptr(), self.n, self.k)

    @staticmethod
    def from_parts(codes: torch.Tensor, scales: torch.Tensor, g_dec: float) -> "NVFP4Weight":
        n, half = codes.shape
        glob = torch.tensor([float(g_dec), 0.0, 0.0, 0.0], dtype=torch.float32, device=codes.device)
        return NVFP4Weight(codes.contiguous(), scales.contiguous(), glob, n, half * 2)


@dataclass
class NVFP4Experts:
    """Stacked routed experts: gate/up codes [E, I, H/2], scales [E, I, H/16];
    down codes [E, H, I/2], scales [E, H, I/16]; globals [E, 4] fp32."""
    gate_codes: torch.Tensor
    gate_scales: torch.Tensor
    gate_glob: torch.Tensor
    up_codes: torch.Tensor
    up_scales: torch.Tensor
    up_glob: torch.Tensor
    down_codes: torch.Tensor
    down_scales: torch.Tensor
    down_glob: torch.Tensor

    @property
    def num_experts(self):
        return self.gate_codes.shape[0]

    @property
    def inter(self):
        return self.gate_codes.shape[1]

    @property
    def hidden(self):
        return self.gate_codes.shape[2] * 2

    def desc(self) -> _MoeWeights:
        return _MoeWeights(self.num_experts, self.hidden, self.inter,
                           self.gate_codes.data_ptr(), self.gate_scales.data_ptr(), self.gate_glob.data_ptr(),
                           self.up_codes.data_ptr(), self.up_scales.data_ptr(), self.up_glob.data_ptr(),
                           self.down_codes.data_ptr(), self.down_scales.data_ptr(), self.down_glob.data_ptr())


def nvfp4_quantize(w: torch.Tensor, out: NVFP4Weight | None = None) -> NVFP4Weight:
    w = _as_bf16(w)
    _dev(w, "w")
    n, k = w.shape
    if out is None:
        dev = w.device
        out = NVFP4Weight(torch.empty((n, k // 2), dtype=torch.uint8, device=dev),
                          torch.empty((n, k // 16), dtype=torch.uint8, device=dev),
                          torch.empty(4, dtype=torch.float32, device=dev), n, k)
    _check(lib().nvfp4_quantize(_ptr(w), n, k, _ptr(out.codes), _ptr(out.scales), _ptr(out.glob), _stream(w)),
           "nvfp4_quantize")
    return out


def _out_code(dtype):
    if dtype == torch.float32:
        return NVFP4_OUT_F32
    if dtype == torch.bfloat16:
        return NVFP4_OUT_BF16
    raise TypeError("output dtype must be float32 or bfloat16")


def w4a16_gemv(x: torch.Tensor, w: NVFP4Weight, out_dtype=torch.float32, out: torch.Tensor | None = None):
    x = _as_bf16(x)
    _dev(x, "x")
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, w.n), dtype=out_dtype, device=x.device)
    d = w.desc()
    _check(lib().w4a16_gemv(_ptr(x), m, ctypes.byref(d), _ptr(out), _out_code(out.dtype), _stream(x)), "w4a16_gemv")
    return out


def w4a16_gemv_embed(idx: torch.Tensor, table: torch.Tensor, x_rest: torch.Tensor | None, w: NVFP4Weight,
                     out_dtype=torch.float32, out: torch.Tensor | None = None):
    """w4a16_gemv over rows [table[idx[i]] | x_rest[i]]: the embedding rows
    of the tokens in idx (int32, e.g. the LM head's out_idx; zero rows for
    ids outside the table) are read by the GEMV itself."""
    _dev(idx, "idx")
    _dev(table, "table")
    if table.dtype != torch.bfloat16 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table must be a contiguous bf16 [vocab][hidden] tensor")
    if idx.dtype != torch.int32 or not idx.is_contiguous():
        raise ValueError("idx must be a contiguous int32 tensor")
    m = idx.numel()
    vocab, hidden = table.shape
    if x_rest is not None:
        x_rest = _as_bf16(x_rest)
        _dev(x_rest, "x_rest")
        if x_rest.shape != (m, w.k - hidden):
            raise ValueError(f"x_rest must be [{m}][{w.k - hidden}]")
    if out is None:
        out = torch.empty((m, w.n), dtype=out_dtype, device=table.device)
    d = w.desc()
    _check(lib().w4a16_gemv_embed(_ptr(idx), _ptr(table), vocab, hidden, _ptr(x_rest), m, ctypes.byref(d), _ptr(out),
                                  _out_code(out.dtype), _stream(table)), "w4a16_gemv_embed")
    return out


def w4a16_gemv_grouped(x: torch.Tensor, ws, out_dtype=torch.float32, outs=None):
    """One launch of the GEMV over several weights with the same K (q|k|v,
    gate|up); returns one output per weight."""
    x = _as_bf16(x)
    _dev(x, "x")
    m = x.shape[0]
    ws = list(ws)
    if outs is None:
        outs = [torch.empty((m, w.n), dtype=out_dtype, device=x.device) for w in ws]
    outs = list(outs)
    if len(outs) != len(ws):
        raise ValueError("w4a16_gemv_grouped: one output per weight")
    code = _out_code(outs[0].dtype) if outs else 0
    for o in outs:
        if _out_code(o.dtype) != code:
            raise ValueError("w4a16_gemv_grouped: all outputs need one dtype")
    descs = [w.desc() for w in ws]
    WP = ctypes.POINTER(_Weight)
    warr = (WP * len(ws))(*[ctypes.pointer(d) for d in descs])
    yarr = (ctypes.c_void_p * len(ws))(*[_ptr(o) for o in outs])
    _check(lib().w4a16_gemv_grouped(_ptr(x), m, warr, yarr, len(ws), code, _stream(x)), "w4a16_gemv_grouped")
    return outs


def gemm_workspace(m: int, n: int, k: int, device) -> torch.Tensor | None:
    """Workspace for w4a16_gemm_m128 at m x n x k on `device` (None when the
    call needs none: its output tiles fill the device)."""
    with torch.cuda.device(device):
        nbytes = lib().w4a16_gemm_m128_workspace_bytes(m, n, k)
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def w4a16_gemm_m128(x: torch.Tensor, w: NVFP4Weight, out_dtype=torch.float32, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, split_k: bool = True):
    """y = x @ W^T.  Short prompt chunks split K over a workspace (allocated
    here when none is given); split_k=False runs one pass over K."""
    x = _as_bf16(x)
    _dev(x, "x")
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, w.n), dtype=out_dtype, device=x.device)
    if split_k and workspace is None:
        workspace = gemm_workspace(m, w.n, w.k, x.device)
    if not split_k:
        workspace = None
    if workspace is not None:
        _dev(workspace, "workspace")
    d = w.desc()
    _check(lib().w4a16_gemm_m128(_ptr(x), m, ctypes.byref(d), _ptr(out), _out_code(out.dtype),
                                 _ptr(workspace) if workspace is not None else None,
                                 workspace.numel() * workspace.element_size() if workspace is not None else 0,
                                 _stream(x)), "w4a16_gemm_m128")
    return out


def lmhead_workspace(m: int, vocab_rows: int, device) -> torch.Tensor:
    """Zero-filled workspace for lmhead_gemv_argmax scoring `vocab_rows` rows
    (the effective V).  It must start zeroed; every call leaves it reusable."""
    nbytes = lib().lmhead_gemv_argmax_workspace_bytes(m, vocab_rows)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def lmhead_gemv_argmax(h: torch.Tensor, w: NVFP4Weight, vocab_rows: int = 0, bf16_keys: bool = False,
                       workspace: torch.Tensor | None = None, out_idx: torch.Tensor | None = None,
                       out_max: torch.Tensor | None = None):
    h = _as_bf16(h)
    _dev(h, "h")
    m = h.shape[0]
    if workspace is None:
        v = w.n if vocab_rows <= 0 else min(vocab_rows, w.n)
        workspace = lmhead_workspace(m, v, h.device)
    if out_idx is None:
        out_idx = torch.empty(m, dtype=torch.int32, device=h.device)
    if out_max is None:
        out_max = torch.empty(m, dtype=torch.float32, device=h.device)
    d = w.desc()
    _check(lib().lmhead_gemv_argmax(_ptr(h), m, ctypes.byref(d), vocab_rows, _ptr(out_idx), _ptr(out_max),
                                    _ptr(workspace), workspace.numel(),
                                    NVFP4_ARGMAX_BF16_KEYS if bf16_keys else 0, _stream(h)),
           "lmhead_gemv_argmax")
    return out_idx, out_max


def lmhead_gemv_argmax_fc(h: torch.Tensor, w: NVFP4Weight, table: torch.Tensor, x_rest: torch.Tensor | None,
                          fc: NVFP4Weight, vocab_rows: int = 0, bf16_keys: bool = False,
                          workspace: torch.Tensor | None = None, out_idx: torch.Tensor | None = None,
                          out_max: torch.Tensor | None = None, out: torch.Tensor | None = None,
                          out_dtype=torch.float32):
    """lmhead_gemv_argmax of h, then the next draft step's fc over the rows
    [table[out_idx[i]] | x_rest[i]] (w4a16_gemv_embed): one launch at one
    row, the two calls otherwise.  Returns (out_idx, out_max, out)."""
    h = _as_bf16(h)
    _dev(h, "h")
    _dev(table, "table")
    if table.dtype != torch.bfloat16 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table must be a contiguous bf16 [vocab][hidden] tensor")
    m = h.shape[0]
    vocab, hidden = table.shape
    if x_rest is not None:
        x_rest = _as_bf16(x_rest)
        _dev(x_rest, "x_rest")
        if x_rest.shape != (m, fc.k - hidden):
            raise ValueError(f"x_rest must be [{m}][{fc.k - hidden}]")
    if workspace is None:
        v = w.n if vocab_rows <= 0 else min(vocab_rows, w.n)
        workspace = lmhead_workspace(m, v, h.device)
    if out_idx is None:
        out_idx = torch.empty(m, dtype=torch.int32, device=h.device)
    if out_max is None:
        out_max = torch.empty(m, dtype=torch.float32, device=h.device)
    if out is None:
        out = torch.empty((m, fc.n), dtype=out_dtype, device=h.device)
    d, dfc = w.desc(), fc.desc()
    _check(lib().lmhead_gemv_argmax_fc(_ptr(h), m, ctypes.byref(d), vocab_rows, _ptr(out_idx), _ptr(out_max),
                                       _ptr(workspace), workspace.numel(), NVFP4_ARGMAX_BF16_KEYS if bf16_keys else 0,
                                       _ptr(table), vocab, hidden, _ptr(x_rest), ctypes.byref(dfc), _ptr(out),
                                       _out_code(out.dtype), _stream(h)),
           "lmhead_gemv_argmax_fc")
    return out_idx, out_max, out


def lmhead_gemv_argmax_noalloc(h: torch.Tensor, w: NVFP4Weight, vocab_rows: int = 0, bf16_keys: bool = False,
                               out_idx: torch.Tensor | None = None, out_max: torch.Tensor | None = None):
    """lmhead_gemv_argmax with the library's static per-device scratch in
    place of a workspace (nothing is allocated by the call itself; pass
    out_idx / out_max to allocate nothing here either).  Calls that overlap
    on one device race."""
    h = _as_bf16(h)
    _dev(h, "h")
    m = h.shape[0]
    if out_idx is None:
        out_idx = torch.empty(m, dtype=torch.int32, device=h.device)
    if out_max is None:
        out_max = torch.empty(m, dtype=torch.float32, device=h.device)
    d = w.desc()
    _check(lib().lmhead_gemv_argmax_noalloc(_ptr(h), m, ctypes.byref(d), vocab_rows, _ptr(out_idx), _ptr(out_max),
                                            NVFP4_ARGMAX_BF16_KEYS if bf16_keys else 0, _stream(h)),
           "lmhead_gemv_argmax_noalloc")
    return out_idx, out_max


def lmhead_gemv_argmax_logprob(h: torch.Tensor, w: NVFP4Weight, vocab_rows: int = 0, bf16_keys: bool = False,
                               workspace: torch.Tensor | None = None, out_idx: torch.Tensor | None = None,
                               out_max: torch.Tensor | None = None, out_logprob: torch.Tensor | None = None):
    """lmhead_gemv_argmax plus the top-1 log-probability of each selected token."""
    h = _as_bf16(h)
    _dev(h, "h")
    m = h.shape[0]
    if workspace is None:
        v = w.n if vocab_rows <= 0 else min(vocab_rows, w.n)
        workspace = lmhead_workspace(m, v, h.device)
    if out_idx is None:
        out_idx = torch.empty(m, dtype=torch.int32, device=h.device)
    if out_max is None:
        out_max = torch.empty(m, dtype=torch.float32, device=h.device)
    if out_logprob is None:
        out_logprob = torch.empty(m, dtype=torch.float32, device=h.device)
    d = w.desc()
    _check(lib().lmhead_gemv_argmax_logprob(_ptr(h), m, ctypes.byref(d), vocab_rows, _ptr(out_idx), _ptr(out_max),
                                            _ptr(out_logprob), _ptr(workspace), workspace.numel(),
                                            NVFP4_ARGMAX_BF16_KEYS if bf16_keys else 0, _stream(h)),
           "lmhead_gemv_argmax_logprob")
    return out_idx, out_max, out_logprob


def lmhead_gemv_argmax_masked(h: torch.Tensor, w: NVFP4Weight, allow_mask: torch.Tensor, vocab_rows: int = 0,
                              bf16_keys: bool = False, with_logprob: bool = False,
                              workspace: torch.Tensor | None = None, out_idx: torch.Tensor | None = None,
                              out_max: torch.Tensor | None = None, out_logprob: torch.Tensor | None = None):
    """Grammar-masked LM-head argmax.  allow_mask: int32/uint32 [m][words] on
    the device (bit r % 32 of word r / 32 allows token r)."""
    h = _as_bf16(h)
    _dev(h, "h")
    _dev(allow_mask, "allow_mask")
    m = h.shape[0]
    if allow_mask.dim() != 2 or allow_mask.shape[0] != m or allow_mask.element_size() != 4:
        raise ValueError("allow_mask must be a [m][words] 32-bit tensor")
    allow_mask = allow_mask.contiguous()
    if workspace is None:
        v = w.n if vocab_rows <= 0 else min(vocab_rows, w.n)
        workspace = lmhead_workspace(m, v, h.device)
    if out_idx is None:
        out_idx = torch.empty(m, dtype=torch.int32, device=h.device)
    if out_max is None:
        out_max = torch.empty(m, dtype=torch.float32, device=h.device)
    if with_logprob and out_logprob is None:
        out_logprob = torch.empty(m, dtype=torch.float32, device=h.device)
    d = w.desc()
    _check(lib().lmhead_gemv_argmax_masked(_ptr(h), m, ctypes.byref(d), vocab_rows, _ptr(allow_mask),
                                           allow_mask.shape[1], _ptr(out_idx), _ptr(out_max), _ptr(out_logprob),
                                           _ptr(workspace), workspace.numel(),
                                           NVFP4_ARGMAX_BF16_KEYS if bf16_keys else 0, _stream(h)),
           "lmhead_gemv_argmax_masked")
    return (out_idx, out_max, out_logprob) if with_logprob else (out_idx, out_max)


def embed_from_argmax(idx: torch.Tensor, table: torch.Tensor, out: torch.Tensor | None = None,
                      id_log: torch.Tensor | None = None):
    """Rows table[idx[i]] of a bf16 [vocab][hidden] table (zero rows for
    out-of-range ids) into out (rows may be strided, e.g. half of a wider
    activation row); id_log, if given, receives the ids."""
    _dev(idx, "idx")
    _dev(table, "table")
    if table.dtype != torch.bfloat16 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table must be a contiguous bf16 [vocab][hidden] tensor")
    m = idx.numel()
    vocab, hidden = table.shape
    if out is None:
        out = torch.empty((m, hidden), dtype=torch.bfloat16, device=table.device)
    if out.dtype != torch.bfloat16 or out.dim() != 2 or out.shape[1] != hidden or out.stride(1) != 1:
        raise ValueError("out must be bf16 [m][hidden] with unit column stride")
    _check(lib().embed_from_argmax(_ptr(idx), m, _ptr(table), vocab, hidden, _ptr(out), out.stride(0), _ptr(id_log),
                                   _stream(table)), "embed_from_argmax")
    return out


def lmhead_gemv_argmax_embed(h: torch.Tensor, w: NVFP4Weight, table: torch.Tensor, out_embed: torch.Tensor,
                             vocab_rows: int = 0, allow_mask: torch.Tensor | None = None, bf16_keys: bool = False,
                             id_log: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                             out_idx: torch.Tensor | None = None, out_max: torch.Tensor | None = None,
                             out_logprob: torch.Tensor | None = None):
    """LM-head argmax whose last workgroup also writes table[idx[i]] into
    out_embed row i (bf16, unit column stride) and idx into id_log."""
    h = _as_bf16(h)
    _dev(h, "h")
    _dev(table, "table")
    m = h.shape[0]
    if table.dtype != torch.bfloat16 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table must be a contiguous bf16 [vocab][hidden] tensor")
    vocab, hidden = table.shape
    if out_embed.dtype != torch.bfloat16 or out_embed.dim() != 2 or out_embed.shape != (m, hidden) \
            or out_embed.stride(1) != 1:
        raise ValueError("out_embed must be bf16 [m][hidden] with unit column stride")
    words = 0
    if allow_mask is not None:
        _dev(allow_mask, "allow_mask")
        allow_mask = allow_mask.contiguous()
        words = allow_mask.shape[1]
    if workspace is None:
        v = w.n if vocab_rows <= 0 else min(vocab_rows, w.n)
        workspace = lmhead_workspace(m, v, h.device)
    if out_idx is None:
        out_idx = torch.empty(m, dtype=torch.int32, device=h.device)
    if out_max is None:
        out_max = torch.empty(m, dtype=torch.float32, device=h.device)
    d = w.desc()
    _check(lib().lmhead_gemv_argmax_embed(_ptr(h), m, ctypes.byref(d), vocab_rows, _ptr(allow_mask), words,
                                          _ptr(out_idx), _ptr(out_max), _ptr(out_logprob), _ptr(table), vocab, hidden,
                                          _ptr(out_embed), out_embed.stride(0), _ptr(id_log), _ptr(workspace),
                                          workspace.numel(), NVFP4_ARGMAX_BF16_KEYS if bf16_keys else 0, _stream(h)),
           "lmhead_gemv_argmax_embed")
    return out_idx, out_max


def moe_workspace(m: int, top_k: int, experts: NVFP4Experts, device) -> torch.Tensor:
    """Zero-filled workspace for moe_w4a16_gemv (must start zeroed; every call
    leaves it reusable)."""
    d = experts.desc()
    nbytes = lib().moe_w4a16_gemv_workspace_bytes(m, top_k, ctypes.byref(d))
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def moe_trace_events(top_k: int, experts: NVFP4Experts) -> tuple[int, int]:
    """(events, workgroups) of a one-token moe_w4a16_gemv_trace: the trace
    holds events x workgroups timestamps, gate/up workgroups first."""
    d = experts.desc()
    words = lib().moe_w4a16_gemv_trace_words(1, top_k, ctypes.byref(d))
    return 6, words // 6


def moe_w4a16_gemv(x: torch.Tensor, router_logits: torch.Tensor, top_k: int, experts: NVFP4Experts,
                   workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   topk_ids: torch.Tensor | None = None, topk_w: torch.Tensor | None = None,
                   trace: torch.Tensor | None = None):
    """Routed MoE over m rows.  With `trace` (int64 [6, workgroups] from
    moe_trace_events, one token only) the one-launch form also records its
    phase timestamps (moe_w4a16_gemv_trace)."""
    x = _as_bf16(x)
    _dev(x, "x")
    _dev(router_logits, "router_logits")
    if router_logits.dtype != torch.float32:
        raise TypeError("router_logits must be float32")
    m = x.shape[0]
    if workspace is None:
        workspace = moe_workspace(m, top_k, experts, x.device)
    if out is None:
        out = torch.empty((m, experts.hidden), dtype=torch.float32, device=x.device)
    if topk_ids is None:
        topk_ids = torch.empty((m, top_k), dtype=torch.int32, device=x.device)
    if topk_w is None:
        topk_w = torch.empty((m, top_k), dtype=torch.float32, device=x.device)
    d = experts.desc()
    if trace is not None:
        _dev(trace, "trace")
        if trace.dtype != torch.int64 or not trace.is_contiguous():
            raise TypeError("trace must be a contiguous int64 tensor")
        _check(lib().moe_w4a16_gemv_trace(_ptr(x), m, _ptr(router_logits), top_k, ctypes.byref(d), _ptr(out),
                                          _ptr(topk_ids), _ptr(topk_w), _ptr(workspace), workspace.numel(),
                                          _ptr(trace), trace.numel(), _stream(x)),
               "moe_w4a16_gemv_trace")
        return out, topk_ids, topk_w
    _check(lib().moe_w4a16_gemv(_ptr(x), m, _ptr(router_logits), top_k, ctypes.byref(d), _ptr(out), _ptr(topk_ids),
                                _ptr(topk_w), _ptr(workspace), workspace.numel(), _stream(x)),
           "moe_w4a16_gemv")
    return out, topk_ids, topk_w


def moe_workspace_status(workspace: torch.Tensor) -> int:
    """Reads and clears the sticky status word of a MoE workspace
    (synchronizes the current stream).  Returns 0; raises NVFP4Error when a
    down pass gave up its wait or found the workspace overwritten."""
    _dev(workspace, "workspace")
    st = ctypes.c_uint32(0)
    _check(lib().moe_workspace_status(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                      ctypes.byref(st), _stream(workspace)), "moe_workspace_status")
    return st.value


def moe_layer_workspace(m: int, top_k: int, experts: NVFP4Experts, device) -> torch.Tensor:
    """Zero-filled workspace for moe_layer_w4a16."""
    d = experts.desc()
    nbytes = lib().moe_layer_w4a16_workspace_bytes(m, top_k, ctypes.byref(d))
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def moe_layer_w4a16(x: torch.Tensor, router: NVFP4Weight, top_k: int, experts: NVFP4Experts,
                    shared_gate: NVFP4Weight, shared_up: NVFP4Weight, shared_down: NVFP4Weight,
                    shared_gate_w: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, topk_ids: torch.Tensor | None = None,
                    topk_w: torch.Tensor | None = None, router_logits: torch.Tensor | None = None):
    """The complete MoE layer; returns (y, topk_ids, topk_w, router_logits)."""
    x = _as_bf16(x)
    _dev(x, "x")
    m = x.shape[0]
    dev = x.device
    if workspace is None:
        workspace = moe_layer_workspace(m, top_k, experts, dev)
    if out is None:
        out = torch.empty((m, experts.hidden), dtype=torch.float32, device=dev)
    if topk_ids is None:
        topk_ids = torch.empty((m, top_k), dtype=torch.int32, device=dev)
    if topk_w is None:
        topk_w = torch.empty((m, top_k), dtype=torch.float32, device=dev)
    if router_logits is None:
        router_logits = torch.empty((m, experts.num_experts), dtype=torch.float32, device=dev)
    if shared_gate_w is not None:
        shared_gate_w = _as_bf16(shared_gate_w).contiguous()
    ds = [w.desc() for w in (router, shared_gate, shared_up, shared_down)]
    d = experts.desc()
    _check(lib().moe_layer_w4a16(_ptr(x), m, ctypes.byref(ds[0]), top_k, ctypes.byref(d), ctypes.byref(ds[1]),
                                 ctypes.byref(ds[2]), ctypes.byref(ds[3]), _ptr(shared_gate_w), _ptr(out),
                                 _ptr(topk_ids), _ptr(topk_w), _ptr(router_logits), _ptr(workspace),
                                 workspace.numel(), _stream(x)), "moe_layer_w4a16")
    return out, topk_ids, topk_w, router_logits



# ---- attention of the draft step over a paged 8-bit cache, and verification
#
# A decode step's kernels take a few microseconds, so these bindings keep the
# host's part short: descriptors of a cache and a batch are made once, pointers
# go to the library as integers, and the device is switched only when it is not
# the current one.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_BF16 = torch.bfloat16


def _run(what: str, fn, index: int, *args):
    """fn(*args, stream) on device `index` and its current stream."""
    if _current_device() == index:      # (a tensor on the device: CUDA is initialised)
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != 0:
        _check(rc, what)


def _int32(t: torch.Tensor, name: str):
    _dev(t, name)
    if t.dtype is not torch.int32:
        raise TypeError(f"{name} must be int32")


def _fits32(v: int, name: str) -> int:
    """A host integer for the library's int32 (ctypes would cut it)."""
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"{name}={v} does not fit 32 bits")
    return v


def _same_device(index: int, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on different devices: cuda:{index} and {t.device}")


def _rows(t: torch.Tensor, name: str) -> _HeadRows:
    """Head rows of a bf16 [rows][heads][dim] tensor (unit stride in dim)."""
    shape = t.shape
    if t.dtype is not _BF16 or len(shape) != 3:
        raise ValueError(f"{name} must be bf16 [rows][heads][dim]")
    n, heads, dim = shape
    row, head, unit = t.stride()
    if unit != 1 and dim != 1:
        raise ValueError(f"{name} must have unit stride in dim")
    return _HeadRows(t.data_ptr(), row if n > 1 else heads * dim, head if heads > 1 else dim, heads, dim)


@dataclass(frozen=True)
class KV8Cache:
    """A paged 8-bit KV cache on the device: k_codes [pages, kv_heads,
    page_tokens, head_dim] and v_codes [pages, kv_heads, head_dim,
    page_tokens] uint8 (E4M3), k_scales and v_scales [pages, kv_heads] uint8
    (byte b stands for 2^(b - 127), at most 2^119).  The tensors keep their
    storage."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor

    def __post_init__(self):
        if self.k_codes.dim() != 4:
            raise ValueError("k_codes must be [pages][kv_heads][page_tokens][head_dim]")
        pages, heads, tokens, dim = self.k_codes.shape
        for t, shape, name in ((self.k_codes, (pages, heads, tokens, dim), "k_codes"),
                               (self.v_codes, (pages, heads, dim, tokens), "v_codes"),
                               (self.k_scales, (pages, heads), "k_scales"), (self.v_scales, (pages, heads), "v_scales")):
            _dev(t, name)
            if t.dtype is not torch.uint8 or t.shape != shape:
                raise ValueError(f"{name} must be uint8 {list(shape)}")
        index = self.k_codes.get_device()
        _same_device(index, self.k_scales, self.v_codes, self.v_scales)
        d = _KV8Cache(self.k_codes.data_ptr(), self.k_scales.data_ptr(), self.v_codes.data_ptr(),
                      self.v_scales.data_ptr(), pages, tokens, heads, dim)
        for name, v in (("index", index), ("kv_heads", heads), ("page_tokens", tokens), ("head_dim", dim), ("_ref", ctypes.byref(d))):
            object.__setattr__(self, name, v)

    @staticmethod
    def empty(num_pages: int, kv_heads: int, head_dim: int, page_tokens: int = 16, device="cuda") -> "KV8Cache":
        def u8(*shape):
            return torch.zeros(shape, dtype=torch.uint8, device=device)
        return KV8Cache(u8(num_pages, kv_heads, page_tokens, head_dim), u8(num_pages, kv_heads),
                        u8(num_pages, kv_heads, head_dim, page_tokens), u8(num_pages, kv_heads))


@dataclass(frozen=True)
class KV8Seqs:
    """A ragged batch over a KV8Cache: cu_rows [batch + 1], kv_lens [batch]
    (this call's rows included) and block_table [batch, max_pages] int32 on
    the device; max_rows bounds a sequence's rows, max_kv_len its length (0:
    what the table holds).  The tensors keep their storage; their values are
    read on the device by every call."""
    cu_rows: torch.Tensor
    kv_lens: torch.Tensor
    block_table: torch.Tensor
    max_rows: int
    max_kv_len: int = 0

    def __post_init__(self):
        batch = self.kv_lens.numel()
        _fits32(self.max_rows, "max_rows")
        _fits32(self.max_kv_len, "max_kv_len")
        for t, name in ((self.cu_rows, "cu_rows"), (self.kv_lens, "kv_lens"), (self.block_table, "block_table")):
            _int32(t, name)
        if self.cu_rows.numel() != batch + 1 or self.block_table.dim() != 2 or self.block_table.shape[0] != batch:
            raise ValueError("need cu_rows [batch + 1], kv_lens [batch], block_table [batch][max_pages]")
        index = self.kv_lens.get_device()
        _same_device(index, self.cu_rows, self.block_table)
        object.__setattr__(self, "index", index)
        object.__setattr__(self, "_refs", {})

    def _ref(self, rows: int):
        ref = self._refs.get(rows)
        if ref is None:
            d = _KV8Seqs(self.cu_rows.data_ptr(), self.kv_lens.data_ptr(), self.block_table.data_ptr(), self.kv_lens.numel(),
                         _fits32(rows, "rows"), self.max_rows, self.block_table.shape[1], self.max_kv_len)
            if len(self._refs) >= 64:
                self._refs.clear()
            ref = self._refs[rows] = ctypes.byref(d)
        return ref


def _rope_desc(inv_freq: torch.Tensor, interleaved: bool, mscale: float) -> _Rope:
    _dev(inv_freq, "inv_freq")
    if inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1:
        raise TypeError("inv_freq must be a float64 vector (rope_frequencies)")
    return _Rope(inv_freq.data_ptr(), 2 * inv_freq.numel(), interleaved, mscale)


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_len: int = 4096, low_turns: float = 1.0, high_turns: float = 32.0, device="cuda"):
    """(inv_freq, mscale) of rope_qk for `rot_dim` rotated elements:
    f_i = base^(-2i / rot_dim), scaled for a context `factor` times
    original_len:
      None        as it is;
      "linear"    f_i / factor (positions squeezed into the trained range);
      "base"      base * factor^(rot_dim / (rot_dim - 2)): the slowest pair is
                  stretched by factor, the fastest not at all;
      "by_parts"  a pair that turns more than high_turns times in original_len
                  is kept, one below low_turns divided by factor, linear in
                  the turns in between; mscale = 1 + 0.1 ln(factor).
    inv_freq is float64 on `device`."""
    if rot_dim < 16 or rot_dim % 16:
        raise ValueError("rot_dim must be a positive multiple of 16")
    if not 0 < base < math.inf or not 1 <= factor < math.inf or not original_len > 0 or \
            not -math.inf < low_turns < high_turns < math.inf:
        raise ValueError("need base > 0, factor >= 1, original_len > 0 and high_turns > low_turns, all finite")
    if scaling not in (None, "linear", "base", "by_parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "base":
        if math.log(base) + math.log(factor) * rot_dim / (rot_dim - 2) > 709.0:
            raise ValueError("the stretched base passes the range of fp64")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    f = torch.exp(-math.log(base) * i / rot_dim)
    mscale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        keep = ((original_len * f / (2 * math.pi) - low_turns) / (high_turns - low_turns)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
        mscale = 0.1 * math.log(factor) + 1.0
    return f.to(device), mscale


def rope_qk(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor,
            interleaved: bool = False, mscale: float = 1.0, q_out: torch.Tensor | None = None,
            k_out: torch.Tensor | None = None):
    """Rotary positions (int32 [rows]) of q and k, bf16 [rows][heads][dim]
    (either may be None; rows and heads may be strided).  Returns (q_out,
    k_out); pass q_out=q to rotate in place."""
    _int32(positions, "positions")
    rows, index, byref = _fits32(positions.numel(), "rows"), positions.get_device(), ctypes.byref
    dq = dqo = dk = dko = None
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        dq, dqo = byref(_rows(q, "q")), byref(_rows(q_out, "q_out"))
        if q.shape[0] != rows or q_out.shape != q.shape:
            raise ValueError(f"q and q_out must have {rows} rows and one shape")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k is not None:
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        dk, dko = byref(_rows(k, "k")), byref(_rows(k_out, "k_out"))
        if k.shape[0] != rows or k_out.shape != k.shape:
            raise ValueError(f"k and k_out must have {rows} rows and one shape")
    elif k_out is not None:
        raise ValueError("k_out without k")
    _same_device(index, q, q_out, k, k_out, inv_freq)
    _run("rope_qk", lib().rope_qk, index, dq, dqo, dk, dko, rows, positions.data_ptr(),
         byref(_rope_desc(inv_freq, interleaved, mscale)))
    return q_out, k_out


def kv8_append(cache: KV8Cache, seqs: KV8Seqs, k: torch.Tensor, v: torch.Tensor):
    """Quantises k and v, bf16 [rows][kv_heads][head_dim], into the cache at
    the rows' positions."""
    if k.shape != v.shape:
        raise ValueError("k and v must have one shape")
    index = cache.index
    _same_device(index, k, v, seqs.kv_lens)
    _run("kv8_append", lib().kv8_append, index, cache._ref, seqs._ref(k.shape[0]), ctypes.byref(_rows(k, "k")),
         ctypes.byref(_rows(v, "v")))


def rope_kv8_append(cache: KV8Cache, seqs: KV8Seqs, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                    inv_freq: torch.Tensor, interleaved: bool = False, mscale: float = 1.0,
                    q_out: torch.Tensor | None = None):
    """rope_qk of q and k at the rows' positions, then kv8_append of the
    rotated k and of v, in one launch.  Returns the rotated q (None without
    q); pass q_out=q to rotate in place."""
    if k.shape != v.shape:
        raise ValueError("k and v must have one shape")
    index, dq, dqo = cache.index, None, None
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if q.shape[0] != k.shape[0] or q_out.shape != q.shape:
            raise ValueError("q and q_out must have k's rows and one shape")
        dq, dqo = ctypes.byref(_rows(q, "q")), ctypes.byref(_rows(q_out, "q_out"))
    elif q_out is not None:
        raise ValueError("q_out without q")
    _same_device(index, q, q_out, k, v, inv_freq, seqs.kv_lens)
    _run("rope_kv8_append", lib().rope_kv8_append, index, cache._ref, seqs._ref(k.shape[0]),
         ctypes.byref(_rope_desc(inv_freq, interleaved, mscale)), dq, dqo, ctypes.byref(_rows(k, "k")),
         ctypes.byref(_rows(v, "v")))
    return q_out


def kv8_read(cache: KV8Cache, seqs: KV8Seqs, rows: int | None = None, k_out: torch.Tensor | None = None,
             v_out: torch.Tensor | None = None):
    """The values of each sequence's last tokens (as many as it owns rows) in
    bf16 [rows][kv_heads][head_dim].  Give the outputs, or `rows` to have both
    allocated here.  Returns (k_out, v_out)."""
    index = cache.index
    if k_out is None and v_out is None:
        if rows is None:
            raise ValueError("kv8_read needs rows, k_out or v_out")
        shape = (rows, cache.kv_heads, cache.head_dim)
        k_out, v_out = (torch.empty(shape, dtype=torch.bfloat16, device=cache.k_codes.device) for _ in range(2))
    elif rows is None:
        rows = (k_out if k_out is not None else v_out).shape[0]
    if (k_out is not None and k_out.shape[0] != rows) or (v_out is not None and v_out.shape[0] != rows):
        raise ValueError(f"outputs must have {rows} rows")
    _same_device(index, k_out, v_out, seqs.kv_lens)
    _run("kv8_read", lib().kv8_read, index, cache._ref, seqs._ref(rows),
         ctypes.byref(_rows(k_out, "k_out")) if k_out is not None else None,
         ctypes.byref(_rows(v_out, "v_out")) if v_out is not None else None)
    return k_out, v_out


def kv8_attention_workspace(cache: KV8Cache, seqs: KV8Seqs, q_heads: int, rows: int) -> torch.Tensor:
    """Workspace for kv8_attention of `rows` rows (nothing to initialise)."""
    _fits32(q_heads, "q_heads")
    with torch.cuda.device(cache.index):
        nbytes = lib().kv8_attention_workspace_bytes(cache._ref, seqs._ref(rows), q_heads)
    if nbytes == 0:
        raise NVFP4Error(lib().nvfp4_mtp_last_error().decode(errors="replace"))
    return torch.empty(nbytes, dtype=torch.uint8, device=cache.k_codes.device)


def kv8_attention(q: torch.Tensor, cache: KV8Cache, seqs: KV8Seqs, scale: float | None = None, window: int = 0,
                  sinks: int = 0, workspace: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """Attention of q, bf16 [rows][q_heads][head_dim], over the cache (scale:
    head_dim^-0.5 by default; 0: a plain mean).  out: bf16
    [rows][q_heads][head_dim], heads contiguous.  Prompt chunks and single rows
    over long caches are faster in two calls than in one."""
    dq, index = _rows(q, "q"), cache.index
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    do = _rows(out, "out")
    if out.shape != q.shape or do.head_stride != do.dim:
        raise ValueError("out must have q's shape and contiguous heads")
    if workspace is None:
        workspace = kv8_attention_workspace(cache, seqs, dq.heads, q.shape[0])
    _dev(workspace, "workspace")
    _same_device(index, q, out, workspace, seqs.kv_lens)
    _run("kv8_attention", lib().kv8_attention, index, ctypes.byref(dq), cache._ref, seqs._ref(q.shape[0]),
         dq.dim ** -0.5 if scale is None else scale, _fits32(window, "window"), _fits32(sinks, "sinks"), do.data, do.row_stride, workspace.data_ptr(),
         workspace.nbytes)
    return out


class Verified(NamedTuple):
    """accepted [batch]: drafts that stand; tokens [rows]: those, the token
    drawn after them, then -1 (rows of no sequence are not written); next [batch]: the drawn token; kv_lens [batch]:
    cache lengths without the fallen drafts' rows (None if not asked for)."""
    accepted: torch.Tensor
    tokens: torch.Tensor
    next: torch.Tensor
    kv_lens: torch.Tensor | None


def verify_workspace(max_rows: int, batch: int, vocab: int, device, sampled: bool = False) -> torch.Tensor:
    """Workspace for verify_drafts (nothing to initialise)."""
    for v, name in ((max_rows, "max_rows"), (batch, "batch"), (vocab, "vocab")):
        _fits32(v, name)
    with torch.cuda.device(device):
        nbytes = lib().verify_drafts_workspace_bytes(batch, max_rows, vocab, int(sampled))
    if nbytes == 0:
        raise NVFP4Error(lib().nvfp4_mtp_last_error().decode(errors="replace"))
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _vector(t: torch.Tensor | None, dtype, n: int, index: int, name: str):
    """The pointer of a contiguous device vector (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous {dtype} on cuda:{index}")
    return t.data_ptr()


def verify_drafts(logits: torch.Tensor, cu_rows: torch.Tensor, draft_ids: torch.Tensor, u_accept: torch.Tensor,
                  u_sample: torch.Tensor, max_rows: int, temperature: torch.Tensor | None = None,
                  draft_logits: torch.Tensor | None = None, kv_lens: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, out: Verified | None = None) -> Verified:
    """Verification of drafted tokens against the target's logits [rows][vocab]
    (fp32 or bf16, rows may be strided), from given random numbers.  Sequence b
    owns rows cu_rows[b] .. cu_rows[b + 1]; draft_ids[r] is the draft after row
    r (a sequence's last row has none).  draft_logits: the rows the drafts were
    sampled from, or None for drafts chosen outright."""
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor")
    index, i32, f32 = logits.get_device(), torch.int32, torch.float32
    _fits32(max_rows, "max_rows")
    rows, vocab = logits.shape
    batch = cu_rows.numel() - 1
    strides = []
    for t, name in ((logits, "logits"), (draft_logits, "draft_logits")):
        if t is None:
            strides.append(0)
            continue
        if t.dtype is not logits.dtype or t.shape != logits.shape or t.get_device() != index or (t.stride(1) != 1 and vocab != 1):
            raise ValueError(f"{name} must have the logits' type, shape and device and unit column stride")
        strides.append(t.stride(0) if rows > 1 else vocab)
    if workspace is None:
        workspace = verify_workspace(max_rows, batch, vocab, logits.device, sampled=draft_logits is not None)
    _dev(workspace, "workspace")
    _same_device(index, workspace)
    if out is None:
        parts = torch.empty(rows + (2 if kv_lens is None else 3) * batch, dtype=i32, device=logits.device) \
            .split_with_sizes([batch, rows, batch] + ([] if kv_lens is None else [batch]))
        out = Verified(*parts, *([None] if kv_lens is None else []))
    _run("verify_drafts", lib().verify_drafts, index, logits.data_ptr(), _out_code(logits.dtype), strides[0], vocab,
         draft_logits.data_ptr() if draft_logits is not None else None, strides[1],
         _vector(cu_rows, i32, batch + 1, index, "cu_rows"), batch, rows, max_rows,
         _vector(draft_ids, i32, rows, index, "draft_ids"), _vector(temperature, f32, batch, index, "temperature"),
         _vector(u_accept, f32, rows, index, "u_accept"), _vector(u_sample, f32, batch, index, "u_sample"),
         _vector(kv_lens, i32, batch, index, "kv_lens"), _vector(out.accepted, i32, batch, index, "out.accepted"),
         _vector(out.tokens, i32, rows, index, "out.tokens"), _vector(out.next, i32, batch, index, "out.next"),
         _vector(out.kv_lens, i32, batch, index, "out.kv_lens"), workspace.data_ptr(), workspace.nbytes)
    return out
