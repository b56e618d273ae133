"""Thin Python binding of ``libpisa.so`` (include/pisa.h), same names as the C ABI.

Argument marshalling only: torch tensors are passed as raw device pointers
together with torch's current CUDA stream; every step of the path runs in the
library's CUDA kernels. If the library is missing or a tensor is not on a CUDA
device, the call raises -- there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpisa.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "pisa.h")

PISA_DTYPE_F32, PISA_DTYPE_BF16 = 0, 1
STATUS = {0: "PISA_OK", -1: "PISA_E_INVALID", -2: "PISA_E_UNSUPPORTED", -3: "PISA_E_CUDA",
          -4: "PISA_E_ALIGNMENT", -5: "PISA_E_TIMEOUT", -6: "PISA_E_SCRATCH_LIMIT"}


class PisaError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({msg})")
        self.status = status


class PisaCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "Hq", "Hkv", "N", "d", "C", "K", "g", "causal", "forced_mask", "dtype", "score_variant")]


class PisaPages(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int32), ("P", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def exported_names() -> list[str]:
    """Function names declared in include/pisa.h."""
    src = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z0-9_]+\s*\*?\s*(pisa_[a-z0-9_]+)\s*\(", src, re.M)))


def load(path: str | None = None):
    """Load libpisa.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if path is None:
            from . import build as _build
            if not _build.up_to_date():  # sources newer than the library: rebuild, never run a stale one
                _build.build()
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with `python -m hierarchical_block_sparse_b200.build`")
        lib = ctypes.CDLL(p)
        P = ctypes.c_void_p
        cfgp = ctypes.POINTER(PisaCfg)
        pgp = ctypes.POINTER(PisaPages)
        I64 = ctypes.c_int64
        sig = {
            "pisa_num_levels": (ctypes.c_int, [cfgp]),
            "pisa_level_nodes": (ctypes.c_int64, [cfgp, ctypes.c_int]),
            "pisa_level_offset": (ctypes.c_int64, [cfgp, ctypes.c_int]),
            "pisa_pyramid_rows": (ctypes.c_int64, [cfgp]),
            "pisa_build_pyramid": (ctypes.c_int, [cfgp, P, P, P]),
            "pisa_select": (ctypes.c_int, [cfgp, P, P, P, P, P]),
            "pisa_sparse_attn": (ctypes.c_int, [cfgp, P, P, P, P, P, P]),
            "pisa_forward": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P]),
            "pisa_bsa_select": (ctypes.c_int, [cfgp, P, P, P, P]),
            "pisa_bsa_select_ws": (ctypes.c_int, [cfgp, P, P, P, P, ctypes.c_size_t, P]),
            "pisa_workspace_bytes": (ctypes.c_int64, [cfgp]),
            "pisa_workspace_status": (ctypes.c_int, [cfgp, P, P]),
            "pisa_select_ws": (ctypes.c_int, [cfgp, P, P, P, P, P, ctypes.c_size_t, P]),
            "pisa_sparse_attn_ws": (ctypes.c_int, [cfgp, P, P, P, P, P, P, ctypes.c_size_t, P]),
            "pisa_forward_ws": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P, ctypes.c_size_t, P]),
            "pisa_forward_host": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]),
            "pisa_forward_ws_events": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P, ctypes.c_size_t,
                                                      ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, P]),
            "pisa_select_noalloc": (ctypes.c_int, [cfgp, P, P, P, P, P]),
            "pisa_select_noalloc_status": (ctypes.c_int, [cfgp, P]),
            "pisa_build_pyramid_prefix": (ctypes.c_int, [cfgp, P, P, P, P]),
            "pisa_pyramid_append": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P]),
            "pisa_pyramid_grow": (ctypes.c_int, [cfgp, P, cfgp, P, P]),
            "pisa_cache_capacity": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int]),
            "pisa_cache_grow": (ctypes.c_int, [cfgp, P, P, P, cfgp, P, P, P, P]),
            "pisa_sparse_attn_backward": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P, P, P]),
            "pisa_backward_workspace_bytes": (ctypes.c_int64, [cfgp]),
            "pisa_sparse_attn_backward_ws": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]),
            "pisa_sparse_attn_backward_saved_ws": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P, P, P, ctypes.c_size_t,
                                                                  P]),
            "pisa_sparse_attn_backward_ws_events": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P, P, P, ctypes.c_size_t,
                                                                   ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, P]),
            "pisa_decode": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P, P]),
            "pisa_decode_step": (ctypes.c_int, [cfgp, P, P, P, P, P, P, P, P, P, P]),
            "pisa_pages_state_words": (I64, [pgp]),
            "pisa_pages_init": (ctypes.c_int, [cfgp, pgp, P, P, P, P]),
            "pisa_pages_reserve": (ctypes.c_int, [cfgp, pgp, P, P, P, P, P, P, I64, P]),
            "pisa_pages_fork": (ctypes.c_int, [cfgp, pgp, P, P, P, P, P, P, P]),
            "pisa_pages_free": (ctypes.c_int, [cfgp, pgp, P, ctypes.c_int, P, P, P, P]),
            "pisa_pages_compact": (ctypes.c_int, [cfgp, pgp, P, P, P, I64, P]),
            "pisa_pages_copy": (ctypes.c_int, [cfgp, pgp, P, I64, P, P, P]),
            "pisa_paged_append": (ctypes.c_int, [cfgp, pgp, P, P, ctypes.c_int, P, P, P, P, P, P]),
            "pisa_paged_workspace_bytes": (I64, [cfgp, pgp]),
            "pisa_paged_attn": (ctypes.c_int, [cfgp, pgp, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]),
            "pisa_paged_build_pyramid": (ctypes.c_int, [cfgp, pgp, P, P, P, P, P]),
            "pisa_paged_pyramid_append": (ctypes.c_int, [cfgp, pgp, P, P, P, P, P, P, P, P]),
            "pisa_paged_decode_step": (ctypes.c_int, [cfgp, pgp, P, P, P, P, P, P, P, P, P, P, P]),
            "pisa_fma_probe": (ctypes.c_int, [P, ctypes.c_int, ctypes.c_int, ctypes.c_int, P]),
            "pisa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "pisa_version": (ctypes.c_char_p, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        if path is None:
            _lib = lib
        return lib


PISA_SCORE_LSE, PISA_SCORE_MEAN, PISA_SCORE_MEAN_VAR = 0, 1, 2


def make_cfg(*, B: int, Hq: int, Hkv: int, N: int, d: int, C: int, K: int, g: int = 2, causal: bool = True,
             forced_mask: int = 7, dtype=torch.bfloat16, score_variant: int = PISA_SCORE_LSE) -> PisaCfg:
    dt = {torch.bfloat16: PISA_DTYPE_BF16, torch.float32: PISA_DTYPE_F32}.get(dtype, dtype)
    return PisaCfg(B, Hq, Hkv, N, d, C, K, g, int(causal), forced_mask, int(dt), int(score_variant))


def cfg_for(Q: torch.Tensor, K: torch.Tensor, *, C: int, K_: int, causal: bool = True, forced_mask: int = 7,
            g: int = 2, score_variant: int = PISA_SCORE_LSE) -> PisaCfg:
    B, Hq, N, d = Q.shape
    return make_cfg(B=B, Hq=Hq, Hkv=K.shape[1], N=N, d=d, C=C, K=K_, g=g, causal=causal,
                    forced_mask=forced_mask, dtype=Q.dtype, score_variant=score_variant)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _host_ptr(t: torch.Tensor):
    if t.is_cuda:
        raise ValueError("host buffers must live in host memory")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(name: str, status: int):
    if status != 0:
        raise PisaError(name, status, load().pisa_status_string(status).decode())


# ---- geometry -------------------------------------------------------------------

def pisa_num_levels(cfg: PisaCfg) -> int:
    return int(load().pisa_num_levels(ctypes.byref(cfg)))


def pisa_level_nodes(cfg: PisaCfg, level: int) -> int:
    return int(load().pisa_level_nodes(ctypes.byref(cfg), level))


def pisa_level_offset(cfg: PisaCfg, level: int) -> int:
    return int(load().pisa_level_offset(ctypes.byref(cfg), level))


def pisa_pyramid_rows(cfg: PisaCfg) -> int:
    r = int(load().pisa_pyramid_rows(ctypes.byref(cfg)))
    if r < 0:
        _check("pisa_pyramid_rows", r)
    return r


# ---- prefill ----------------------------------------------------------------------

def pisa_build_pyramid(cfg, K, pyr):
    _check("pisa_build_pyramid", load().pisa_build_pyramid(ctypes.byref(cfg), _ptr(K), _ptr(pyr), _stream()))


def pisa_select(cfg, Q, K, pyr, idx):
    _check("pisa_select", load().pisa_select(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(pyr), _ptr(idx), _stream()))


def pisa_sparse_attn(cfg, Q, K, V, idx, O):
    _check("pisa_sparse_attn", load().pisa_sparse_attn(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx),
                                                       _ptr(O), _stream()))


def pisa_forward(cfg, Q, K, V, pyr, idx, O):
    _check("pisa_forward", load().pisa_forward(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(pyr), _ptr(idx),
                                               _ptr(O), _stream()))


def pisa_bsa_select(cfg, Q, pyr, idx):
    _check("pisa_bsa_select", load().pisa_bsa_select(ctypes.byref(cfg), _ptr(Q), _ptr(pyr), _ptr(idx), _stream()))


def pisa_bsa_select_ws(cfg, Q, pyr, idx, ws):
    """Flat BSA selection (Eq.1) on the tensor cores, in the block-major workspace."""
    _check("pisa_bsa_select_ws", load().pisa_bsa_select_ws(ctypes.byref(cfg), _ptr(Q), _ptr(pyr), _ptr(idx),
                                                           _ptr(ws), ws.numel(), _stream()))


# ---- block-major tensor-core prefill (workspace) -----------------------------------

def pisa_workspace_bytes(cfg) -> int:
    r = int(load().pisa_workspace_bytes(ctypes.byref(cfg)))
    if r < 0:
        _check("pisa_workspace_bytes", r)
    return r


def alloc_workspace(cfg, device="cuda") -> torch.Tensor:
    """Caller-owned workspace for the *_ws calls (torch allocates; 256-byte aligned)."""
    return torch.empty(max(pisa_workspace_bytes(cfg), 256), dtype=torch.uint8, device=device)


def pisa_workspace_status(cfg, ws) -> int:
    """0, or -5 (PISA_E_TIMEOUT) when a tensor-core tile gave up a bounded wait (synchronises)."""
    return int(load().pisa_workspace_status(ctypes.byref(cfg), _ptr(ws), _stream()))


def pisa_select_ws(cfg, Q, K, pyr, idx, ws):
    _check("pisa_select_ws", load().pisa_select_ws(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(pyr), _ptr(idx),
                                                   _ptr(ws), ws.numel(), _stream()))


def pisa_sparse_attn_ws(cfg, Q, K, V, idx, O, ws):
    _check("pisa_sparse_attn_ws", load().pisa_sparse_attn_ws(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V),
                                                             _ptr(idx), _ptr(O), _ptr(ws), ws.numel(), _stream()))


def pisa_forward_ws(cfg, Q, K, V, pyr, idx, O, ws):
    _check("pisa_forward_ws", load().pisa_forward_ws(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(pyr),
                                                     _ptr(idx), _ptr(O), _ptr(ws), ws.numel(), _stream()))


def pisa_forward_host(cfg, Q_host, K_host, V_host, idx_host, O_host, Q, K, V, pyr, idx, O, ws):
    """pisa_forward_ws from host buffers (pinned for asynchronous copies) on the current stream."""
    _check("pisa_forward_host", load().pisa_forward_host(
        ctypes.byref(cfg), _host_ptr(Q_host), _host_ptr(K_host), _host_ptr(V_host), _host_ptr(idx_host),
        _host_ptr(O_host), _ptr(Q), _ptr(K), _ptr(V), _ptr(pyr), _ptr(idx), _ptr(O), _ptr(ws), ws.numel(),
        _stream()))


def pisa_select_noalloc(cfg, Q, K, pyr, idx):
    """pisa_select_ws without a workspace: for callers that cannot allocate device
    memory, the library's fixed 32 MiB scratch array is used instead (calls on a
    device share it, so they must not overlap on the GPU)."""
    _check("pisa_select_noalloc", load().pisa_select_noalloc(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(pyr),
                                                             _ptr(idx), _stream()))


def pisa_select_noalloc_status(cfg) -> int:
    """Error word of the last pisa_select_noalloc on this device: 0, or -5
    (PISA_E_TIMEOUT) when a tile gave up a bounded wait or a self-check failed
    (synchronises the current stream)."""
    return int(load().pisa_select_noalloc_status(ctypes.byref(cfg), _stream()))


def pisa_fma_probe(out, blocks: int, iters: int, packed: bool):
    """Launch the fp32 FMA throughput probe on the current stream (out: fp32, blocks * 256 elements)."""
    assert out.numel() >= blocks * 256 and out.dtype == torch.float32
    _check("pisa_fma_probe", load().pisa_fma_probe(_ptr(out), int(blocks), int(iters), int(bool(packed)),
                                                   _stream()))


PHASES = ["pyramid", "stage1", "group_candidates", "leaf_scores", "topk", "group_kept", "forced_tiles",
          "attn_tiles", "finalize"]


def pisa_forward_ws_events(cfg, Q, K, V, pyr, idx, O, ws, events):
    """pisa_forward_ws recording torch.cuda.Event objects (len(PHASES) + 1) at phase boundaries."""
    stream = torch.cuda.current_stream()
    for e in events:
        if e.cuda_event == 0:  # torch creates the underlying event on first record
            e.record(stream)
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check("pisa_forward_ws_events", load().pisa_forward_ws_events(
        ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(pyr), _ptr(idx), _ptr(O), _ptr(ws), ws.numel(),
        arr, len(events), _stream()))


# ---- decode -------------------------------------------------------------------------

def pisa_build_pyramid_prefix(cfg, Kc, length, pyr):
    _check("pisa_build_pyramid_prefix", load().pisa_build_pyramid_prefix(ctypes.byref(cfg), _ptr(Kc), _ptr(length),
                                                                         _ptr(pyr), _stream()))


def pisa_pyramid_append(cfg, Kc, Vc, pyr, k_new, v_new, pos):
    _check("pisa_pyramid_append", load().pisa_pyramid_append(ctypes.byref(cfg), _ptr(Kc), _ptr(Vc), _ptr(pyr),
                                                             _ptr(k_new), _ptr(v_new), _ptr(pos), _stream()))


def pisa_sparse_attn_backward(cfg, Q, K, V, idx, dO, dQ, dK, dV):
    """dQ, dK, dV (fp32) of the sparse attention for the fixed selection idx."""
    _check("pisa_sparse_attn_backward", load().pisa_sparse_attn_backward(
        ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx), _ptr(dO), _ptr(dQ), _ptr(dK), _ptr(dV), _stream()))


def pisa_backward_workspace_bytes(cfg) -> int:
    r = int(load().pisa_backward_workspace_bytes(ctypes.byref(cfg)))
    if r < 0:
        _check("pisa_backward_workspace_bytes", r)
    return r


def alloc_backward_workspace(cfg, device="cuda") -> torch.Tensor:
    """Caller-owned workspace for pisa_sparse_attn_backward_ws (256-byte aligned)."""
    return torch.empty(max(pisa_backward_workspace_bytes(cfg), 256), dtype=torch.uint8, device=device)


def pisa_sparse_attn_backward_ws(cfg, Q, K, V, idx, dO, dQ, dK, dV, ws):
    """pisa_sparse_attn_backward, block-major on the tensor cores (bf16, d = 128, C = 64)."""
    _check("pisa_sparse_attn_backward_ws", load().pisa_sparse_attn_backward_ws(
        ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx), _ptr(dO), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(ws),
        ws.numel(), _stream()))


def pisa_sparse_attn_backward_saved_ws(cfg, Q, K, V, idx, dO, dQ, dK, dV, ws):
    """The backward reusing what pisa_forward_ws / pisa_sparse_attn_ws left in ws (same inputs)."""
    _check("pisa_sparse_attn_backward_saved_ws", load().pisa_sparse_attn_backward_saved_ws(
        ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx), _ptr(dO), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(ws),
        ws.numel(), _stream()))


BWD_PHASES = ["statistics", "zeroing", "backward_tiles"]


def pisa_sparse_attn_backward_ws_events(cfg, Q, K, V, idx, dO, dQ, dK, dV, ws, events):
    """pisa_sparse_attn_backward_ws recording torch.cuda.Event objects (len(BWD_PHASES) + 1)."""
    stream = torch.cuda.current_stream()
    for e in events:
        if e.cuda_event == 0:
            e.record(stream)
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check("pisa_sparse_attn_backward_ws_events", load().pisa_sparse_attn_backward_ws_events(
        ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx), _ptr(dO), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(ws),
        ws.numel(), arr, len(events), _stream()))


def pisa_pyramid_grow(cfg_old, pyr_old, cfg_new, pyr_new):
    _check("pisa_pyramid_grow", load().pisa_pyramid_grow(ctypes.byref(cfg_old), _ptr(pyr_old), ctypes.byref(cfg_new),
                                                         _ptr(pyr_new), _stream()))


def pisa_cache_capacity(n: int, C: int) -> int:
    """The library's geometric capacity for n cached keys (smallest C * 2^k >= n)."""
    r = int(load().pisa_cache_capacity(int(n), int(C)))
    if r < 0:
        _check("pisa_cache_capacity", r)
    return r


def pisa_cache_grow(cfg_old, Kc_old, Vc_old, pyr_old, cfg_new, Kc_new, Vc_new, pyr_new):
    _check("pisa_cache_grow", load().pisa_cache_grow(ctypes.byref(cfg_old), _ptr(Kc_old), _ptr(Vc_old), _ptr(pyr_old),
                                                     ctypes.byref(cfg_new), _ptr(Kc_new), _ptr(Vc_new),
                                                     _ptr(pyr_new), _stream()))


class DecodeCache:
    """K and V caches [B, Hkv, capacity, d] and their pyramid, grown by the
    library's geometric policy: before a step would write at or past the
    capacity, buffers of pisa_cache_capacity(needed) rows are allocated (torch)
    and pisa_cache_grow moves the contents. cfg.N is the capacity. The
    per-sequence positions stay in the caller's pos tensor."""

    def __init__(self, cfg, Kc: torch.Tensor, Vc: torch.Tensor, pyr: torch.Tensor):
        self.cfg, self.Kc, self.Vc, self.pyr = cfg, Kc, Vc, pyr

    @property
    def capacity(self) -> int:
        return int(self.cfg.N)

    def reserve(self, n: int) -> None:
        """Make room for n keys per sequence (grows geometrically when needed)."""
        if n <= self.cfg.N:
            return
        c = self.cfg
        new = PisaCfg(c.B, c.Hq, c.Hkv, pisa_cache_capacity(n, c.C), c.d, c.C, c.K, c.g, c.causal, c.forced_mask,
                      c.dtype, c.score_variant)
        shape = (c.B, c.Hkv, new.N, c.d)
        # growing writes every row of the new buffers, except from an empty cache (nothing to move)
        alloc = torch.zeros if c.N == 0 else torch.empty
        Kc = alloc(shape, dtype=self.Kc.dtype, device=self.Kc.device)
        Vc = alloc(shape, dtype=self.Vc.dtype, device=self.Vc.device)
        pyr = alloc((c.B, c.Hkv, pisa_pyramid_rows(new), c.d), dtype=torch.float32, device=self.pyr.device)
        pisa_cache_grow(c, self.Kc, self.Vc, self.pyr, new, Kc, Vc, pyr)
        self.cfg, self.Kc, self.Vc, self.pyr = new, Kc, Vc, pyr

    def step(self, q_new, k_new, v_new, pos, idx, o, max_pos: int) -> None:
        """pisa_decode_step for every sequence, growing first if the largest
        position (max_pos, a host value: no device read) reaches the capacity."""
        self.reserve(max_pos + 1)
        pisa_decode_step(self.cfg, q_new, k_new, v_new, self.Kc, self.Vc, self.pyr, pos, idx, o)


def pisa_decode(cfg, q_new, Kc, Vc, pyr, pos, idx, o):
    _check("pisa_decode", load().pisa_decode(ctypes.byref(cfg), _ptr(q_new), _ptr(Kc), _ptr(Vc), _ptr(pyr),
                                             _ptr(pos), _ptr(idx), _ptr(o), _stream()))


def pisa_decode_step(cfg, q_new, k_new, v_new, Kc, Vc, pyr, pos, idx, o):
    _check("pisa_decode_step", load().pisa_decode_step(ctypes.byref(cfg), _ptr(q_new), _ptr(k_new), _ptr(v_new),
                                                       _ptr(Kc), _ptr(Vc), _ptr(pyr), _ptr(pos), _ptr(idx), _ptr(o),
                                                       _stream()))


# ---- paged decode cache ---------------------------------------------------------------

def make_pages(S: int, P: int) -> PisaPages:
    """S tokens per page, P pages in the pool."""
    return PisaPages(int(S), int(P))


def pages_width(cfg, pages) -> int:
    """W: table entries per sequence."""
    return -(-cfg.N // pages.S)


def pisa_pages_state_words(pages) -> int:
    r = int(load().pisa_pages_state_words(ctypes.byref(pages)))
    if r < 0:
        _check("pisa_pages_state_words", r)
    return r


def _elem(cfg):
    return torch.bfloat16 if cfg.dtype == PISA_DTYPE_BF16 else torch.float32


def _state_words(pages):
    P = pages.P
    return 2 * (P + 3 & ~3) + 3 * ((P + 31) // 32 + 3 & ~3) + 16


# These calls are made at every token: one check and one pointer a tensor, no lists.

def _dev(t) -> int:
    d = t.get_device()
    if d < 0:
        raise ValueError("tensors must live on a CUDA device")
    return d


def _at(t, dtype, n, dev):
    """The address of t, which holds at least n elements of dtype on device dev."""
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous() or t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        if t.get_device() != dev:
            raise ValueError(f"tensors on different devices ({dev}, {t.get_device()})")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        raise ValueError(f"expected at least {n} elements of {dtype}, got {t.numel()} of {t.dtype}")
    return t.data_ptr()


def _token(t, dtype, n, dev):
    """The address of a token's rows a sequence, [B, Hkv, d] or [B, Hkv, 1, d]."""
    if t.dim() == 4 and t.shape[2] != 1:
        raise ValueError(f"expected one row a sequence, got {t.shape[2]}")
    return _at(t, dtype, n, dev)


def _go(dev, fn, *args) -> None:
    """fn on device dev and its current stream."""
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status != 0:
        _check(fn.__name__, status)


_i32 = torch.int32


def pisa_pages_init(cfg, pages, state, table, lens):
    """An empty cache: every page free, table -1, lengths 0."""
    dev, B = _dev(state), cfg.B
    _go(dev, (_lib or load()).pisa_pages_init, cfg, pages, _at(state, _i32, _state_words(pages), dev),
        _at(table, _i32, B * -(-cfg.N // pages.S), dev), _at(lens, _i32, B, dev))


def pisa_pages_reserve(cfg, pages, add, state, table, lens, grant, moves):
    """Room for add[b] more tokens of each sequence; lens grows by grant[b]."""
    dev, B = _dev(state), cfg.B
    _go(dev, (_lib or load()).pisa_pages_reserve, cfg, pages, _at(add, _i32, B, dev),
        _at(state, _i32, _state_words(pages), dev), _at(table, _i32, B * -(-cfg.N // pages.S), dev),
        _at(lens, _i32, B, dev), _at(grant, _i32, B, dev), _at(moves, _i32, 4, dev), moves.numel())


def pisa_pages_fork(cfg, pages, parent, state, table, lens, table_out, lens_out):
    """Sequence b becomes a copy of sequence parent[b] (outside [0, B): it ends), sharing its pages."""
    dev, B = _dev(state), cfg.B
    n = B * -(-cfg.N // pages.S)
    _go(dev, (_lib or load()).pisa_pages_fork, cfg, pages, _at(parent, _i32, B, dev),
        _at(state, _i32, _state_words(pages), dev), _at(table, _i32, n, dev), _at(lens, _i32, B, dev),
        _at(table_out, _i32, n, dev), _at(lens_out, _i32, B, dev))


def pisa_pages_free(cfg, pages, seqs, state, table, lens):
    """Ends the listed sequences."""
    dev, B = _dev(state), cfg.B
    _go(dev, (_lib or load()).pisa_pages_free, cfg, pages, _at(seqs, _i32, 0, dev), seqs.numel(),
        _at(state, _i32, _state_words(pages), dev), _at(table, _i32, B * -(-cfg.N // pages.S), dev),
        _at(lens, _i32, B, dev))


def pisa_pages_compact(cfg, pages, state, table, moves):
    """Moves the live pages to the low end of the pool; `moves` lists the copies to make."""
    dev = _dev(state)
    _go(dev, (_lib or load()).pisa_pages_compact, cfg, pages, _at(state, _i32, _state_words(pages), dev),
        _at(table, _i32, cfg.B * -(-cfg.N // pages.S), dev), _at(moves, _i32, 4, dev), moves.numel())


def pisa_pages_copy(cfg, pages, moves, K, V):
    """Copies the pages of one layer as `moves` lists them."""
    dev, dt = _dev(moves), _elem(cfg)
    n = pages.P * pages.S * cfg.Hkv * cfg.d
    _go(dev, (_lib or load()).pisa_pages_copy, cfg, pages, _at(moves, _i32, 4, dev), moves.numel(), _at(K, dt, n, dev),
        _at(V, dt, n, dev))


def _new_rows(k_new, v_new) -> int:
    """T: rows a sequence that are to be appended."""
    T = k_new.shape[2] if k_new.dim() == 4 else 1
    if v_new.dim() == 4 and v_new.shape[2] != T:
        raise ValueError(f"k_new and v_new differ in rows a sequence ({T}, {v_new.shape[2]})")
    return T


def pisa_paged_append(cfg, pages, k_new, v_new, lens, count, table, K, V):
    """Writes rows k_new[b, :, i], v_new[b, :, i] ([B, Hkv, T, d], or [B, Hkv, d]), i < count[b], as the
    last count[b] of the sequence's lens[b] tokens."""
    dev, dt, B, S = _dev(K), _elem(cfg), cfg.B, pages.S
    row = cfg.Hkv * cfg.d
    T = _new_rows(k_new, v_new)
    _go(dev, (_lib or load()).pisa_paged_append, cfg, pages, _at(k_new, dt, B * T * row, dev),
        _at(v_new, dt, B * T * row, dev), T, _at(lens, _i32, B, dev), _at(count, _i32, B, dev),
        _at(table, _i32, B * -(-cfg.N // S), dev), _at(K, dt, pages.P * S * row, dev), _at(V, dt, pages.P * S * row, dev))


def pisa_paged_workspace_bytes(cfg, pages) -> int:
    r = int(load().pisa_paged_workspace_bytes(ctypes.byref(cfg), ctypes.byref(pages)))
    if r < 0:
        _check("pisa_paged_workspace_bytes", r)
    return r


def alloc_paged_workspace(cfg, pages, device="cuda") -> torch.Tensor:
    """Caller-owned workspace for pisa_paged_attn."""
    return torch.empty(pisa_paged_workspace_bytes(cfg, pages), dtype=torch.uint8, device=device)


def pisa_paged_attn(cfg, pages, q, k_new, v_new, K, V, table, lens, o, lse, ws):
    """Dense attention of one token a sequence over its paged cache (k_new, v_new given: appended on the way)."""
    dev, dt, B, S, d = _dev(K), _elem(cfg), cfg.B, pages.S, cfg.d
    rows, row = B * cfg.Hq, cfg.Hkv * d
    n = pages.P * S * row
    _go(dev, (_lib or load()).pisa_paged_attn, cfg, pages, _at(q, dt, rows * d, dev),
        None if k_new is None else _token(k_new, dt, B * row, dev), None if v_new is None else _token(v_new, dt, B * row, dev),
        _at(K, dt, n, dev), _at(V, dt, n, dev), _at(table, _i32, B * -(-cfg.N // S), dev), _at(lens, _i32, B, dev),
        _at(o, dt, rows * d, dev), None if lse is None else _at(lse, torch.float32, rows, dev),
        _at(ws, torch.uint8, 0, dev), ws.numel())


def pisa_paged_build_pyramid(cfg, pages, K, table, lens, pyr):
    """pisa_build_pyramid_prefix from a paged cache; sequences with lens[b] <= 0 are left untouched."""
    dev, B, S, row = _dev(K), cfg.B, pages.S, cfg.Hkv * cfg.d
    _go(dev, (_lib or load()).pisa_paged_build_pyramid, cfg, pages, _at(K, _elem(cfg), pages.P * S * row, dev),
        _at(table, _i32, B * -(-cfg.N // S), dev), _at(lens, _i32, B, dev),
        _at(pyr, torch.float32, B * row * pisa_pyramid_rows(cfg), dev))


def pisa_paged_pyramid_append(cfg, pages, k_new, v_new, K, V, table, lens, pyr):
    """One token's rows into the pages (token lens[b] - 1) and into the summaries."""
    dev, dt, B, S, row = _dev(K), _elem(cfg), cfg.B, pages.S, cfg.Hkv * cfg.d
    n = pages.P * S * row
    _go(dev, (_lib or load()).pisa_paged_pyramid_append, cfg, pages, _token(k_new, dt, B * row, dev), _token(v_new, dt, B * row, dev),
        _at(K, dt, n, dev), _at(V, dt, n, dev), _at(table, _i32, B * -(-cfg.N // S), dev), _at(lens, _i32, B, dev),
        _at(pyr, torch.float32, B * row * pisa_pyramid_rows(cfg), dev))


def pisa_paged_decode_step(cfg, pages, q_new, k_new, v_new, K, V, table, lens, pyr, idx, o):
    """pisa_decode_step over a paged cache; the token in hand is token lens[b] - 1."""
    dev, dt, B, S, d = _dev(K), _elem(cfg), cfg.B, pages.S, cfg.d
    heads = cfg.Hkv
    row, qn = heads * d, B * cfg.Hq * d
    n = pages.P * S * row
    _go(dev, (_lib or load()).pisa_paged_decode_step, cfg, pages, _at(q_new, dt, qn, dev), _token(k_new, dt, B * row, dev),
        _token(v_new, dt, B * row, dev), _at(K, dt, n, dev), _at(V, dt, n, dev), _at(table, _i32, B * -(-cfg.N // S), dev),
        _at(lens, _i32, B, dev), _at(pyr, torch.float32, B * row * pisa_pyramid_rows(cfg), dev),
        _at(idx, _i32, B * heads * cfg.K, dev), _at(o, dt, qn, dev))


class PagedCache:
    """A decode cache in pages: pools K, V [P, Hkv, S, d] and, for the sparse step, a
    pyramid, for each layer; one table, lengths and page state for all of them.
    cfg.N is the most tokens a sequence may hold. No call reads device memory on
    the host; `moves[1]` (pages missing at the last reserve) is for the caller to read.
    Every tensor keeps its address, so graphs captured from these calls can be replayed
    between any others, forks included.
    A sequence that was granted nothing at the last reserve, or was forked or freed since, has
    no token in hand: `step`, and `attend` with new rows, write nothing for it and give it
    o = 0 (idx = -1, lse = -inf).
    A sparse cache whose pages hold whole leaves (S % C == 0) keeps the summaries of every layer
    with all that is written, so a layer's tokens may be attended densely at first and sparsely later
    (layers that never step are better kept in a cache with sparse=False: one launch less a token)."""

    def __init__(self, cfg, pages, layers: int = 1, sparse: bool = True, device="cuda"):
        self.cfg, self.pages = cfg, pages
        dt, W = _elem(cfg), pages_width(cfg, pages)
        shape = (pages.P, cfg.Hkv, pages.S, cfg.d)
        i32 = dict(dtype=torch.int32, device=device)
        self.K = [torch.empty(shape, dtype=dt, device=device) for _ in range(layers)]
        self.V = [torch.empty(shape, dtype=dt, device=device) for _ in range(layers)]
        self.pyr = [torch.empty((cfg.B, cfg.Hkv, pisa_pyramid_rows(cfg), cfg.d), dtype=torch.float32, device=device)
                    for _ in range(layers if sparse else 0)]
        self._sums = sparse and pages.S % cfg.C == 0   # pages hold whole leaves: there are summaries to keep
        self.state = torch.empty(pisa_pages_state_words(pages), **i32)
        # table and lengths in one buffer, which the cache keeps for life (captured graphs hold its
        # address); fork writes the other and copies it back
        self._ints, self._forked = torch.zeros(cfg.B * (W + 1), **i32), torch.zeros(cfg.B * (W + 1), **i32)
        self.table, self.lens = self._ints[:cfg.B * W].view(cfg.B, W), self._ints[cfg.B * W:]
        self._hand = torch.zeros((2, cfg.B), **i32)
        self.grant, self.now = self._hand  # the tokens granted last; lens of the sequences that got some, else 0
        self.moves = torch.zeros(4 + 2 * max(cfg.B, pages.P // 2), **i32)
        self.ws = alloc_paged_workspace(cfg, pages, device)
        pisa_pages_init(cfg, pages, self.state, self.table, self.lens)

    def _copy(self) -> None:
        for K, V in zip(self.K, self.V):
            pisa_pages_copy(self.cfg, self.pages, self.moves, K, V)

    def reserve(self, add: torch.Tensor) -> torch.Tensor:
        """Room for add[b] more tokens; returns grant (the tokens each sequence got)."""
        pisa_pages_reserve(self.cfg, self.pages, add, self.state, self.table, self.lens, self.grant, self.moves)
        torch.mul(self.lens, self.grant > 0, out=self.now)
        self._copy()
        return self.grant

    def append(self, k_new, v_new, layer: int = 0, count: torch.Tensor | None = None) -> None:
        """Rows of the tokens granted last (or of `count`) into the pages. A sparse cache's summaries
        follow: of one token in its own leaf and ancestors, of several by a build of the sequences that got them."""
        count = self.grant if count is None else count
        T = _new_rows(k_new, v_new)
        if self._sums and T > 0:
            _at(count, _i32, self.cfg.B, self.lens.get_device())
            first = count.view(-1)[:self.cfg.B]
            lens = self.lens * ((first > 0) & (first <= T))   # of the sequences that get rows
        if self._sums and T == 1:
            pisa_paged_pyramid_append(self.cfg, self.pages, k_new, v_new, self.K[layer], self.V[layer], self.table, lens,
                                      self.pyr[layer])
            return
        pisa_paged_append(self.cfg, self.pages, k_new, v_new, self.lens, count, self.table, self.K[layer], self.V[layer])
        if self._sums and T > 1:
            self.build_pyramid(layer, lens)

    def build_pyramid(self, layer: int = 0, lens: torch.Tensor | None = None) -> None:
        """Summaries of what is cached (or of lens[b] tokens; <= 0: left as they are, so `now` means the
        sequences of the last reserve). The other calls keep them; rows written past the class need this."""
        pisa_paged_build_pyramid(self.cfg, self.pages, self.K[layer], self.table, self.lens if lens is None else lens,
                                 self.pyr[layer])

    def attend(self, q, o, lse=None, k_new=None, v_new=None, layer: int = 0) -> None:
        """Dense attention of one token a sequence (its rows appended on the way when given; a sparse
        cache's summaries follow, so that steps can)."""
        if self._sums and k_new is not None and v_new is not None:
            pisa_paged_pyramid_append(self.cfg, self.pages, k_new, v_new, self.K[layer], self.V[layer], self.table, self.now,
                                      self.pyr[layer])
            pisa_paged_attn(self.cfg, self.pages, q, None, None, self.K[layer], self.V[layer], self.table, self.now, o, lse, self.ws)
            return
        pisa_paged_attn(self.cfg, self.pages, q, k_new, v_new, self.K[layer], self.V[layer], self.table,
                        self.lens if k_new is None else self.now, o, lse, self.ws)

    def step(self, q_new, k_new, v_new, idx, o, layer: int = 0) -> None:
        """The sparse step (append, select, attend) for the token reserved last."""
        pisa_paged_decode_step(self.cfg, self.pages, q_new, k_new, v_new, self.K[layer], self.V[layer], self.table,
                               self.now, self.pyr[layer], idx, o)

    def fork(self, parent: torch.Tensor) -> None:
        """Sequence b becomes a copy of sequence parent[b]; pyramids of the new ones are rebuilt.
        No sequence has a token in hand then: rows are written again behind the next reserve."""
        n = self.table.numel()
        pisa_pages_fork(self.cfg, self.pages, parent, self.state, self.table, self.lens, self._forked[:n], self._forked[n:])
        self._ints.copy_(self._forked)
        self._hand.zero_()
        if self._sums:
            same = parent == torch.arange(self.cfg.B, dtype=torch.int32, device=parent.device)
            lens = self.lens.masked_fill(same, 0)
            for layer in range(len(self.pyr)):
                self.build_pyramid(layer, lens)

    def free(self, seqs: torch.Tensor) -> None:
        """Ends the listed sequences."""
        pisa_pages_free(self.cfg, self.pages, seqs, self.state, self.table, self.lens)

    def compact(self) -> None:
        """Moves the live pages of every layer to the low end of the pools."""
        pisa_pages_compact(self.cfg, self.pages, self.state, self.table, self.moves)
        self._copy()


def pisa_status_string(status: int) -> str:
    return load().pisa_status_string(status).decode()


def pisa_version() -> str:
    return load().pisa_version().decode()


# ---- allocation helpers (torch owns the memory) --------------------------------------

def alloc_outputs(cfg: PisaCfg, device="cuda", dtype=torch.bfloat16):
    """pyr (fp32), idx (int32) and O tensors sized for cfg."""
    R = pisa_pyramid_rows(cfg)
    pyr = torch.empty((cfg.B, cfg.Hkv, R, cfg.d), dtype=torch.float32, device=device)
    idx = torch.empty((cfg.B, cfg.Hkv, cfg.N, cfg.K), dtype=torch.int32, device=device)
    O = torch.empty((cfg.B, cfg.Hq, cfg.N, cfg.d), dtype=dtype, device=device)
    return pyr, idx, O


def forward(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, *, C: int, K_: int, causal: bool = True,
            forced_mask: int = 7):
    """Allocate outputs and run pisa_forward. Returns (O, idx, pyr)."""
    cfg = cfg_for(Q, K, C=C, K_=K_, causal=causal, forced_mask=forced_mask)
    pyr, idx, O = alloc_outputs(cfg, Q.device, Q.dtype)
    pisa_forward(cfg, Q, K, V, pyr, idx, O)
    return O, idx, pyr
