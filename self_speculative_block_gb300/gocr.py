"""ctypes binding of libgocr.so (include/gocr.h): argument marshalling only.

Every step of the decode path runs in the library's CUDA kernels.  PyTorch
provides device memory (the allocator callback and the weight tensors) and the
CUDA stream; nothing here computes.  When the library has not been built the
import of a decoder fails loudly: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, List, NamedTuple, Optional, Sequence

import numpy as np

from . import synth

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgocr.so")

GOCR_OK = 0
ERRORS = {-1: "EINVAL", -2: "ECAPACITY", -3: "ECUDA", -4: "EDEVICE", -5: "ETIMEOUT",
          -6: "ENOMEM", -7: "ESTATE"}
DTYPE_F32, DTYPE_BF16 = 0, 1
MODE_AR, MODE_SELFSPEC, MODE_DIFFUSION, MODE_REFINED = 0, 1, 2, 3
FWD_AR, FWD_DRAFT, FWD_VERIFY = 0, 1, 2
OPT_ATTENTION, OPT_ATTN_RANKS = 5, 6
TRACE_KERNELS, TRACE_CTAS = 1, 2
TRACE_CTA_SLOTS = 2048
ATTN_TCGEN05, ATTN_MMA_SYNC = 0, 1
MAX_BLOCK = 64
LAYER_TENSORS = 9

# every symbol include/gocr.h declares
EXPORTS = ("gocr_create", "gocr_prefill", "gocr_decode", "gocr_decode_batch", "gocr_decode_ex",
           "gocr_set_draft_override", "gocr_debug_forward", "gocr_debug_forward_batch", "gocr_read_kv", "gocr_get_state",
           "gocr_get_option", "gocr_read_trace", "gocr_last_error", "gocr_free",
           "gocr_op_linear_workspace", "gocr_op_linear", "gocr_op_linear_planes", "gocr_op_attention",
           "gocr_op_linear_static", "gocr_op_attention_ranges", "gocr_three_stream_ranges",
           "gocr_op_embed", "gocr_op_embed_backward_workspace", "gocr_op_embed_backward",
           "gocr_op_linear_ce_workspace", "gocr_op_linear_ce", "gocr_op_linear_ce_backward_workspace",
           "gocr_op_linear_ce_backward", "gocr_op_linear_ce_backward_with_loss", "gocr_op_attention_packed", "gocr_op_attention_packed_backward_workspace",
           "gocr_op_attention_packed_backward", "gocr_op_page_step", "gocr_op_kv_write_paged",
           "gocr_op_attention_paged_workspace", "gocr_op_attention_paged", "gocr_op_status", "gocr_op_wait_probe")


class GocrError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERRORS.get(code, code)}: {msg}")
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("ffn", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("rms_eps", ctypes.c_float),
                ("rope_theta", ctypes.c_float), ("max_ctx", ctypes.c_int32),
                ("max_block", ctypes.c_int32), ("max_requests", ctypes.c_int32),
                ("eos_id", ctypes.c_int32)]


class Weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("mask_embed", ctypes.c_void_p),
                ("lm_head", ctypes.c_void_p), ("g_final", ctypes.c_void_p),
                ("layer", ctypes.POINTER(ctypes.c_void_p))]


class Stats(ctypes.Structure):
    _fields_ = [("rounds", ctypes.c_int64), ("forwards", ctypes.c_int64),
                ("committed", ctypes.c_int64), ("accepted_drafts", ctypes.c_int64),
                ("accept_hist", ctypes.c_int32 * (MAX_BLOCK + 1)), ("device_ms", ctypes.c_double)]

    def as_dict(self) -> dict:
        d = {k: getattr(self, k) for k in ("rounds", "forwards", "committed", "accepted_drafts",
                                           "device_ms")}
        d["accept_hist"] = list(self.accept_hist)
        d["tpf"] = self.committed / self.forwards if self.forwards else 0.0
        return d


class PagedKV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_page", ctypes.c_int64), ("k_head", ctypes.c_int64), ("k_token", ctypes.c_int64),
                ("v_page", ctypes.c_int64), ("v_head", ctypes.c_int64), ("v_token", ctypes.c_int64),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class DecodeOpts(ctypes.Structure):
    _fields_ = [("tau", ctypes.c_float), ("draft_steps", ctypes.c_int32), ("temperature", ctypes.c_float),
                ("reserved", ctypes.c_uint32), ("seed", ctypes.c_uint64)]


ALLOC_FN = ctypes.CFUNCTYPE(ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p)
FREE_FN = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_void_p)

_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Open the library (built by __graft_entry__.build() or build.py)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libgocr.so is not built ({path}); run the package build first")
    lib = ctypes.CDLL(path)
    vp, i32, sz, f32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_longlong
    P32 = ctypes.POINTER(ctypes.c_int32)
    sig = {
        "gocr_create": (i32, [ctypes.POINTER(Config), ctypes.POINTER(Weights), vp, ALLOC_FN, FREE_FN, vp,
                              ctypes.POINTER(vp)]),
        "gocr_prefill": (i32, [vp, i32, vp, i32]),
        "gocr_decode": (i32, [vp, i32, i32, i32, i32, P32, ctypes.POINTER(Stats)]),
        "gocr_decode_batch": (i32, [vp, i32, P32, i32, i32, P32, ctypes.POINTER(P32),
                                    ctypes.POINTER(Stats)]),
        "gocr_decode_ex": (i32, [vp, i32, P32, i32, i32, ctypes.POINTER(DecodeOpts), P32, ctypes.POINTER(P32),
                                 ctypes.POINTER(Stats)]),
        "gocr_set_draft_override": (i32, [vp, i32, P32, i32, P32, i32]),
        "gocr_debug_forward": (i32, [vp, i32, i32, P32, i32, ctypes.POINTER(ctypes.c_float)]),
        "gocr_debug_forward_batch": (i32, [vp, i32, P32, i32, P32, i32, ctypes.POINTER(ctypes.c_float)]),
        "gocr_read_kv": (i32, [vp, i32, i32, i32, i32, vp, vp]),
        "gocr_get_state": (i32, [vp, i32, P32, P32]),
        "gocr_read_trace": (i32, [vp, i32, vp, sz]),
        "gocr_get_option": (i32, [vp, i32, P32]),
        "gocr_last_error": (ctypes.c_char_p, [vp]),
        "gocr_free": (None, [vp]),
        "gocr_op_linear_workspace": (sz, [i32, i32, i32]),
        "gocr_op_linear": (i32, [i32, vp, vp, vp, i32, i32, i32, vp, sz, vp]),
        "gocr_op_linear_planes": (i32, [vp, vp, vp, vp, i32, i32, i32, vp, sz, ctypes.c_uint, vp]),
        "gocr_op_attention": (i32, [i32, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]),
        "gocr_op_linear_static": (i32, [i32, vp, vp, vp, i32, i32, i32, vp]),
        "gocr_op_attention_ranges": (i32, [i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]),
        "gocr_three_stream_ranges": (i32, [i32, i32, i32, P32, P32, P32, P32]),
        "gocr_op_embed": (i32, [i32, vp, vp, vp, vp, i32, i32, i32, f32, vp]),
        "gocr_op_embed_backward_workspace": (sz, [i32, i32]),
        "gocr_op_embed_backward": (i32, [i32, vp, vp, vp, vp, i32, i32, i32, f32, vp, sz, vp]),
        "gocr_op_linear_ce_workspace": (sz, [i32, i32]),
        "gocr_op_linear_ce": (i32, [vp, vp, vp, vp, vp, i32, i32, i32, vp, sz, vp]),
        "gocr_op_linear_ce_backward_workspace": (sz, [i32, i32, i32]),
        "gocr_op_linear_ce_backward": (i32, [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, sz, vp]),
        "gocr_op_linear_ce_backward_with_loss": (i32, [vp] * 8 + [i32, i32, i32, vp, sz, vp]),
        "gocr_op_attention_packed": (i32, [vp] * 6 + [i32] * 5 + [i64] * 3 + [f32, vp]),
        "gocr_op_attention_packed_backward_workspace": (sz, [i32, i32]),
        "gocr_op_attention_packed_backward": (i32, [vp] * 10 + [i32] * 5 + [i64] * 3 + [f32, vp, sz, vp]),
        "gocr_op_page_step": (i32, [vp] * 3 + [i32, vp, i32, i32, vp, i32] + [vp] * 7 + [i32, vp]),
        "gocr_op_kv_write_paged": (i32, [vp] * 6 + [ctypes.POINTER(PagedKV), i32, i32, i64, i64, i64, f32, vp]),
        "gocr_op_attention_paged_workspace": (sz, [i32] * 4),
        "gocr_op_attention_paged": (i32, [vp, ctypes.POINTER(PagedKV), vp, i32, vp, vp, i32, vp, vp, i32, i32, i32, i64,
                                          f32, vp, sz, vp]),
        "gocr_op_status": (i32, [vp]),
        "gocr_op_wait_probe": (i32, [i32, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def last_error(h=None) -> str:
    s = load().gocr_last_error(h)
    return s.decode() if s else ""


def _check(rc: int, h=None):
    if rc != GOCR_OK:
        raise GocrError(rc, last_error(h))


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _p32(a: np.ndarray):
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


# ----------------------------------------------------------------------------
# torch plumbing (device memory and streams only)
# ----------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def to_device(a: np.ndarray, dtype: str, device):
    """Host array (fp32 values, or bf16 bit patterns) -> device tensor in dtype."""
    torch = _torch()
    if dtype == synth.BF16:
        bits = a if a.dtype == np.uint16 else synth.bf16_bits(a)
        return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device)


class _TorchAllocator:
    """Device allocations for the library, served by torch's caching allocator."""

    def __init__(self, device):
        self.device = device
        self.live: Dict[int, object] = {}
        self.alloc_cb = ALLOC_FN(self._alloc)
        self.free_cb = FREE_FN(self._free)

    def _alloc(self, nbytes, _user):
        torch = _torch()
        try:
            t = torch.empty(int(nbytes), dtype=torch.uint8, device=self.device)
        except Exception:
            return None
        p = t.data_ptr()
        self.live[p] = t
        return p

    def _free(self, ptr, _user):
        self.live.pop(int(ptr or 0), None)


class Decoder:
    """One handle: a synthetic decoder resident on one GPU plus its KV caches."""

    def __init__(self, cfg: synth.ModelConfig, weights: dict, max_ctx: int, max_block: int = 32,
                 max_requests: int = 1, eos_id: int = -1, device: str = "cuda:0",
                 use_torch_alloc: bool = True):
        torch = _torch()
        self.lib = load()
        self.cfg = cfg
        self.device = torch.device(device)
        self.max_ctx, self.max_block, self.max_requests = max_ctx, max_block, max_requests
        dt = cfg.dtype
        with torch.cuda.device(self.device):
            self._keep: List[object] = []

            def up(a, d=dt):
                t = to_device(a, d, self.device)
                self._keep.append(t)
                return t.data_ptr()

            ptrs = []
            for lw in weights["layers"]:
                for name in synth.LAYER_MATS:
                    ptrs.append(up(lw[name]))
                ptrs.append(up(lw["g_attn"], synth.F32))
                ptrs.append(up(lw["g_mlp"], synth.F32))
            self._layer_ptrs = (ctypes.c_void_p * len(ptrs))(*ptrs)
            w = Weights(up(weights["embed"]), up(weights["mask_embed"]), up(weights["lm_head"]),
                        up(weights["g_final"], synth.F32),
                        ctypes.cast(self._layer_ptrs, ctypes.POINTER(ctypes.c_void_p)))
            c = Config(cfg.n_layers, cfg.hidden, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim, cfg.ffn,
                       cfg.vocab, DTYPE_BF16 if dt == synth.BF16 else DTYPE_F32, cfg.rms_eps,
                       cfg.rope_theta, max_ctx, max_block, max_requests, eos_id)
            self._alloc = _TorchAllocator(self.device) if use_torch_alloc else None
            h = ctypes.c_void_p()
            stream = torch.cuda.current_stream(self.device).cuda_stream
            rc = self.lib.gocr_create(ctypes.byref(c), ctypes.byref(w), stream,
                                      self._alloc.alloc_cb if self._alloc else ALLOC_FN(),
                                      self._alloc.free_cb if self._alloc else FREE_FN(), None,
                                      ctypes.byref(h))
            _check(rc, None)
            self.h = h

    # ------------------------------------------------------------------ calls
    def close(self):
        if getattr(self, "h", None):
            self.lib.gocr_free(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prefill(self, req: int, prefix) -> None:
        """prefix: host array [P, hidden] (values of cfg.dtype) or a device tensor."""
        torch = _torch()
        if isinstance(prefix, np.ndarray):
            if self.cfg.dtype == synth.BF16:
                host = np.ascontiguousarray(prefix if prefix.dtype == np.uint16 else synth.bf16_bits(prefix))
            else:
                host = np.ascontiguousarray(prefix, dtype=np.float32)
            _check(self.lib.gocr_prefill(self.h, req, host.ctypes.data, host.shape[0]), self.h)
        else:
            assert isinstance(prefix, torch.Tensor) and prefix.is_contiguous()
            _check(self.lib.gocr_prefill(self.h, req, prefix.data_ptr(), prefix.shape[0]), self.h)

    def decode(self, req: int, mode: int, B: int, max_new: int, out: Optional[np.ndarray] = None):
        out = np.zeros(max_new, np.int32) if out is None else out
        st = Stats()
        _check(self.lib.gocr_decode(self.h, req, mode, B, max_new, _p32(out), ctypes.byref(st)), self.h)
        return out, st.as_dict()

    def decode_batch(self, reqs: Sequence[int], mode: int, B: int, max_new: Sequence[int]):
        n = len(reqs)
        r = _i32(reqs)
        mn = _i32(max_new)
        outs = [np.zeros(int(m), np.int32) for m in max_new]
        optr = (ctypes.POINTER(ctypes.c_int32) * n)(*[_p32(o) for o in outs])
        sts = (Stats * n)()
        _check(self.lib.gocr_decode_batch(self.h, n, _p32(r), mode, B, _p32(mn), optr, sts), self.h)
        return outs, [s.as_dict() for s in sts]

    def decode_ex(self, reqs: Sequence[int], mode: int, B: int, max_new: Sequence[int], tau: float = 0.0,
                  draft_steps: int = 1, temperature: float = 0.0, seed: int = 0):
        """Any decode mode over several requests; MODE_DIFFUSION takes the
        confidence threshold tau, MODE_REFINED the draft-side threshold tau and
        at most draft_steps draft forwards per round; MODE_AR and MODE_SELFSPEC
        sample at temperature > 0 with the random-number key seed."""
        n = len(reqs)
        r = _i32(reqs)
        mn = _i32(max_new)
        outs = [np.zeros(int(m), np.int32) for m in max_new]
        optr = (ctypes.POINTER(ctypes.c_int32) * n)(*[_p32(o) for o in outs])
        sts = (Stats * n)()
        opts = DecodeOpts(float(tau), int(draft_steps), float(temperature), 0, int(seed))
        _check(self.lib.gocr_decode_ex(self.h, n, _p32(r), mode, B, ctypes.byref(opts), _p32(mn), optr, sts),
               self.h)
        return outs, [s.as_dict() for s in sts]

    def set_draft_override(self, req: int, ref: Sequence[int], schedule: Sequence[int]):
        ref_a = _i32(ref)
        sch = _i32(schedule)
        _check(self.lib.gocr_set_draft_override(self.h, req, _p32(ref_a), len(ref_a), _p32(sch),
                                                len(sch)), self.h)

    def clear_draft_override(self, req: int):
        z = np.zeros(1, np.int32)
        _check(self.lib.gocr_set_draft_override(self.h, req, _p32(z), 0, _p32(z), 0), self.h)

    def debug_forward(self, req: int, kind: int, tokens: Sequence[int]) -> np.ndarray:
        t = _i32(tokens)
        logits = np.zeros((len(t), self.cfg.vocab), np.float32)
        _check(self.lib.gocr_debug_forward(self.h, req, kind, _p32(t), len(t),
                                           logits.ctypes.data_as(ctypes.POINTER(ctypes.c_float))),
               self.h)
        return logits

    def debug_forward_batch(self, reqs: Sequence[int], kind: int, tokens) -> np.ndarray:
        """One batched forward over several requests; tokens [n_req, n]; logits [n_req, n, vocab]."""
        r = _i32(reqs)
        t = _i32(tokens)
        n_req, n = t.shape
        logits = np.zeros((n_req, n, self.cfg.vocab), np.float32)
        _check(self.lib.gocr_debug_forward_batch(self.h, n_req, _p32(r), kind, _p32(t.reshape(-1)), n,
                                                 logits.ctypes.data_as(ctypes.POINTER(ctypes.c_float))), self.h)
        return logits

    def read_kv(self, req: int, layer: int, pos0: int, n: int):
        """Cached K (rotated) and V of positions pos0..pos0+n-1: two fp32 arrays [n, Hkv, d]."""
        shape = (n, self.cfg.n_kv_heads, self.cfg.head_dim)
        k = np.zeros(shape, np.float32)
        v = np.zeros(shape, np.float32)
        _check(self.lib.gocr_read_kv(self.h, req, layer, pos0, n, k.ctypes.data, v.ctypes.data), self.h)
        return k, v

    def attention_kind(self) -> int:
        """ATTN_TCGEN05 or ATTN_MMA_SYNC, fixed at create time (by chunks per rank, or GOCR_ATTN=tc | mma)."""
        return self._option(OPT_ATTENTION)

    def attention_ranks(self) -> int:
        """Key-chunk ranks of the handle's attention (fixed at create time)."""
        return self._option(OPT_ATTN_RANKS)

    def _option(self, opt: int) -> int:
        v = ctypes.c_int32()
        _check(self.lib.gocr_get_option(self.h, opt, ctypes.byref(v)), self.h)
        return v.value

    def read_kernel_trace(self) -> np.ndarray:
        """Per-launch timeline of the last debug forward run with one kernel per
        operation: uint64 [5 L + 1, 8] (first start, first and last dependency
        release, last end, last mainloop end, last split-K exchange end; ns)."""
        out = np.zeros((5 * self.cfg.n_layers + 1, 8), np.uint64)
        _check(self.lib.gocr_read_trace(self.h, TRACE_KERNELS, out.ctypes.data, out.size), self.h)
        return out

    def read_cta_trace(self) -> np.ndarray:
        """Per-CTA timelines of the last debug forward (GOCR_OP_TRACE=2 at
        create): uint64 [5 L + 1, 2048, 8]; CTA c of a launch in slot c, the
        attention merge kernel's CTAs from slot 1024; zero where unreached."""
        out = np.zeros((5 * self.cfg.n_layers + 1, TRACE_CTA_SLOTS, 8), np.uint64)
        _check(self.lib.gocr_read_trace(self.h, TRACE_CTAS, out.ctypes.data, out.size), self.h)
        return out

    def state(self, req: int):
        cl = ctypes.c_int32()
        x0 = ctypes.c_int32()
        _check(self.lib.gocr_get_state(self.h, req, ctypes.byref(cl), ctypes.byref(x0)), self.h)
        return cl.value, x0.value


# ----------------------------------------------------------------------------
# single-kernel calls on torch tensors
# ----------------------------------------------------------------------------

def _dt(t) -> int:
    torch = _torch()
    return DTYPE_BF16 if t.dtype == torch.bfloat16 else DTYPE_F32


def op_linear(x, w, workspace=None):
    """y[T, N] fp32 = x[T, K] w[N, K]^T through the decoder's split-K GEMM."""
    torch = _torch()
    lib = load()
    T, K = x.shape
    N = w.shape[0]
    y = torch.empty((T, N), dtype=torch.float32, device=x.device)
    need = lib.gocr_op_linear_workspace(T, N, K)
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=x.device)
    stream = torch.cuda.current_stream(x.device).cuda_stream
    _check(lib.gocr_op_linear(_dt(x), x.data_ptr(), w.data_ptr(), y.data_ptr(), T, N, K,
                              workspace.data_ptr(), workspace.numel(), stream))
    return y


OP_OVERLAP = 1


def op_linear_planes(x_hi, x_lo, w, workspace=None, flags: int = 0):
    """y[T, N] fp32 = (x_hi + x_lo)[T, K] w[N, K]^T on bf16 planes, the
    decoder's GEMM on its activation planes.  flags=OP_OVERLAP launches it as
    the decoder does (programmatic dependent launch; w must not be written by
    the stream's previous kernel)."""
    torch = _torch()
    lib = load()
    T, K = x_hi.shape
    N = w.shape[0]
    if x_lo.shape != x_hi.shape or not (x_hi.dtype == x_lo.dtype == w.dtype == torch.bfloat16):
        raise ValueError("op_linear_planes takes bf16 planes of one shape and bf16 weights")
    y = torch.empty((T, N), dtype=torch.float32, device=x_hi.device)
    need = lib.gocr_op_linear_workspace(T, N, K)
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=x_hi.device)
    stream = torch.cuda.current_stream(x_hi.device).cuda_stream
    _check(lib.gocr_op_linear_planes(x_hi.data_ptr(), x_lo.data_ptr(), w.data_ptr(), y.data_ptr(), T, N, K,
                                     workspace.data_ptr(), workspace.numel(), flags, stream))
    return y


def op_linear_static(x, w):
    """op_linear without a workspace: the library's static device scratch array
    (for callers that cannot allocate device memory)."""
    torch = _torch()
    lib = load()
    T, K = x.shape
    N = w.shape[0]
    y = torch.empty((T, N), dtype=torch.float32, device=x.device)
    with torch.cuda.device(x.device):  # the library takes the scratch address of the current device
        stream = torch.cuda.current_stream(x.device).cuda_stream
        _check(lib.gocr_op_linear_static(_dt(x), x.data_ptr(), w.data_ptr(), y.data_ptr(), T, N, K, stream))
    return y


def three_stream_ranges(P: int, N: int, B: int):
    """Row key intervals (lim, lo2, hi2) and rotary positions of the joint
    training mask over [prefix, clean, corrupted 1, corrupted 2] (host int32
    arrays of P + 3 N), from the library."""
    n = P + 3 * N
    lim, lo2, hi2, pos = (np.zeros(n, np.int32) for _ in range(4))
    _check(load().gocr_three_stream_ranges(P, N, B, _p32(lim), _p32(lo2), _p32(hi2), _p32(pos)))
    return lim, lo2, hi2, pos


def op_attention(q, kc, vc, lim, dtype: int, lo2=None, hi2=None):
    """The decoder's attention kernel for `dtype` (DTYPE_BF16 / DTYPE_F32).

    q [T, Hq, d], kc and vc [Hkv, cap, d]: fp32 tensors for DTYPE_F32, or
    (hi, lo) pairs of bf16 tensors for DTYPE_BF16; lim int32 [T] on the
    device; lo2, hi2 (optional) int32 [T] on the device: a second key
    interval per row.  Returns fp32 [T, Hq, d]."""
    torch = _torch()
    lib = load()
    pair = lambda t: (t[0], t[1]) if isinstance(t, (tuple, list)) else (t, None)
    (qh, ql), (kh, kl), (vh, vl) = pair(q), pair(kc), pair(vc)
    T, Hq, d = qh.shape
    Hkv, cap, _ = kh.shape
    o = torch.empty((T, Hq, d), dtype=torch.float32, device=qh.device)
    ptr = lambda t: t.data_ptr() if t is not None else None
    stream = torch.cuda.current_stream(qh.device).cuda_stream
    _check(lib.gocr_op_attention_ranges(dtype, ptr(qh), ptr(ql), ptr(kh), ptr(kl), ptr(vh), ptr(vl), o.data_ptr(),
                                        lim.data_ptr(), ptr(lo2), ptr(hi2), T, Hq, Hkv, d, cap, stream))
    return o


# ----------------------------------------------------------------------------
# training and scoring operators (outside autograd: each has a call for its gradient)
# ----------------------------------------------------------------------------

def _want(name: str, t, shape: tuple, dtype, device):
    """Check one operand: a contiguous CUDA tensor of this shape, dtype and device."""
    if t.dtype == dtype and t.shape == shape and t.is_contiguous() and t.device == device:
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, the other operands are on {device}")


def _lead(name: str, t, dims: int, *dtypes):
    """Check the type and rank of the operand that the others follow."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must be a tensor of {dims} dimensions, got {list(t.shape)}")


def _ready(device, sizes, *operands) -> None:
    """The last checks before device work.  Sizes go to the library as 32-bit
    numbers, which would be cut silently; the calls build no autograd graph, so an
    operand that wants a gradient would lose it silently."""
    bits = 0
    for n in sizes:
        bits |= n
    if bits >> 31:
        raise ValueError(f"a size of {list(sizes)} is outside 0 .. 2^31 - 1")
    for t in operands:
        if t is not None and t.requires_grad and _torch().is_grad_enabled():
            raise ValueError("an operand requires grad, but these calls are outside autograd: detach it, or call "
                             "under torch.no_grad(), and use the _backward calls")
    if device.type != "cuda":
        raise ValueError(f"the operands must be CUDA tensors, got {device}")


def _launch(device, fn, *args) -> None:
    """Call a C entry on the device's current stream, with the device current."""
    torch = _torch()
    index = device.index
    current = getattr(torch._C, "_cuda_getDevice", None)  # (a CUDA tensor in hand: CUDA is initialised)
    if (current() if current is not None else torch.cuda.current_device()) != index:
        with torch.cuda.device(index):
            return _check(fn(*args, torch.cuda.current_stream().cuda_stream))
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without building a Stream object
    _check(fn(*args, raw(index) if raw is not None else torch.cuda.current_stream().cuda_stream))


def _workspace(ws, need: int, device):
    torch = _torch()
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    _want("workspace", ws, (ws.numel(),), torch.uint8, device)
    return ws


def op_embed(ids, embed, mask_embed=None, scale: float = 1.0):
    """y[T, H] = scale * the rows of embed [V, H] (bf16 or fp32) that ids (int32
    [T]) name; id -1 is the [M] row mask_embed [H] (zero without one), any
    other id outside the table a row of zeros."""
    torch = _torch()
    _lead("embed", embed, 2, torch.bfloat16, torch.float32)
    dev, (V, H), T = embed.device, embed.shape, ids.numel()
    _want("embed", embed, (V, H), embed.dtype, dev)
    _want("ids", ids, (T,), torch.int32, dev)
    if mask_embed is not None:
        _want("mask_embed", mask_embed, (H,), embed.dtype, dev)
    _ready(dev, (T, H, V), embed, mask_embed)
    y = torch.empty((T, H), dtype=embed.dtype, device=dev)
    _launch(dev, load().gocr_op_embed, _dt(embed), embed.data_ptr(), mask_embed.data_ptr() if mask_embed is not None
            else None, ids.data_ptr(), y.data_ptr(), T, H, V, scale)
    return y


def op_embed_backward(dy, ids, vocab: int, scale: float = 1.0, mask: bool = False, workspace=None):
    """Gradient of op_embed from dy [T, H]: (d_embed [vocab, H], d_mask [H] when
    mask else None), dense, in dy's dtype, fp32 sums in a fixed order."""
    torch = _torch()
    lib = load()
    _lead("dy", dy, 2, torch.bfloat16, torch.float32)
    dev, (T, H) = dy.device, dy.shape
    _want("dy", dy, (T, H), dy.dtype, dev)
    _want("ids", ids, (T,), torch.int32, dev)
    _ready(dev, (T, H, vocab), dy)
    d_embed = torch.empty((vocab, H), dtype=dy.dtype, device=dev)
    d_mask = torch.empty((H,), dtype=dy.dtype, device=dev) if mask else None
    ws = _workspace(workspace, lib.gocr_op_embed_backward_workspace(T, H), dev)
    _launch(dev, lib.gocr_op_embed_backward, _dt(dy), dy.data_ptr(), ids.data_ptr(), d_embed.data_ptr(),
            d_mask.data_ptr() if mask else None, T, H, vocab, scale, ws.data_ptr(), ws.numel())
    return d_embed, d_mask


def _rows(name: str, t, T, heads, d, device):
    """Check a [T, heads, d] bf16 operand whose rows may lie apart; returns the row pitch."""
    torch = _torch()
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != T or shape[2] != d or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [{T}, {'*' if heads is None else heads}, {d}], got {list(shape)}")
    if stride[2] != 1 or (shape[1] > 1 and stride[1] != d):
        raise ValueError(f"the heads of a row of {name} must be contiguous, got strides {stride}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, q is on {device}")
    return stride[0] if T > 1 else shape[1] * d


def _packed_args(q, k, v, cu_seqlens, scale):
    torch = _torch()
    _lead("q", q, 3, torch.bfloat16)
    dev, (T, Hq, d) = q.device, q.shape
    ld = [_rows("q", q, T, None, d, dev), _rows("k", k, T, None, d, dev)]
    ld.append(_rows("v", v, T, k.shape[1], d, dev))
    n = cu_seqlens.numel()
    _want("cu_seqlens", cu_seqlens, (n,), torch.int32, dev)
    if n < 1:
        raise ValueError("cu_seqlens must hold at least one entry")
    sizes = (n - 1, T, Hq, k.shape[1], d, *ld, d ** -0.5 if scale is None else scale)
    return dev, T, Hq, k.shape[1], d, sizes


def op_attention_packed(q, k, v, cu_seqlens, scale=None, o=None, lse=None):
    """Causal attention over packed sequences with grouped heads: q [T, Hq, d],
    k and v [T, Hkv, d] bf16 (rows may be views of one fused projection);
    sequence s is rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1 (int32, on the
    device); scale defaults to 1 / sqrt(d).  Returns (o [T, Hq, d] bf16, lse
    [Hq, T] fp32), written into o and lse when given; rows of no sequence are
    not written."""
    torch = _torch()
    dev, T, Hq, Hkv, d, sizes = _packed_args(q, k, v, cu_seqlens, scale)
    _ready(dev, sizes[:5], q, k, v)
    if o is None:
        o = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=dev)
    else:
        _want("o", o, (T, Hq, d), torch.bfloat16, dev)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
    else:
        _want("lse", lse, (Hq, T), torch.float32, dev)
    _launch(dev, load().gocr_op_attention_packed, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
            lse.data_ptr(), cu_seqlens.data_ptr(), *sizes)
    return o, lse


def op_attention_packed_backward(do, q, k, v, o, lse, cu_seqlens, scale=None, workspace=None, dq=None, dk=None,
                                 dv=None):
    """Gradient of op_attention_packed from do [T, Hq, d] and the forward
    call's o and lse: (dq [T, Hq, d], dk, dv [T, Hkv, d]) bf16, written into
    dq, dk and dv when given; rows of no sequence are not written."""
    torch = _torch()
    lib = load()
    dev, T, Hq, Hkv, d, sizes = _packed_args(q, k, v, cu_seqlens, scale)
    _want("do", do, (T, Hq, d), torch.bfloat16, dev)
    _want("o", o, (T, Hq, d), torch.bfloat16, dev)
    _want("lse", lse, (Hq, T), torch.float32, dev)
    _ready(dev, sizes[:5], do, q, k, v, o, lse)
    out = []
    for name, t, heads in (("dq", dq, Hq), ("dk", dk, Hkv), ("dv", dv, Hkv)):
        if t is None:
            t = torch.empty((T, heads, d), dtype=torch.bfloat16, device=dev)
        else:
            _want(name, t, (T, heads, d), torch.bfloat16, dev)
        out.append(t)
    ws = _workspace(workspace, lib.gocr_op_attention_packed_backward_workspace(T, Hq), dev)
    _launch(dev, lib.gocr_op_attention_packed_backward, do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
            o.data_ptr(), lse.data_ptr(), cu_seqlens.data_ptr(), out[0].data_ptr(), out[1].data_ptr(),
            out[2].data_ptr(), *sizes, ws.data_ptr(), ws.numel())
    return tuple(out)


def op_linear_ce(x, w, labels, workspace=None):
    """(loss [T], lse [T]) fp32 of the softmax cross entropy of x w^T: x [T, H]
    and w [V, H] bf16, labels int32 [T] (outside 0..V-1: no target, loss 0).
    The logits are not stored."""
    torch = _torch()
    lib = load()
    _lead("x", x, 2, torch.bfloat16)
    dev, (T, H), V = x.device, x.shape, w.shape[0]
    _want("x", x, (T, H), torch.bfloat16, dev)
    _want("w", w, (V, H), torch.bfloat16, dev)
    _want("labels", labels, (T,), torch.int32, dev)
    _ready(dev, (T, V, H), x, w)
    loss = torch.empty((T,), dtype=torch.float32, device=dev)
    lse = torch.empty((T,), dtype=torch.float32, device=dev)
    ws = _workspace(workspace, lib.gocr_op_linear_ce_workspace(T, V), dev)
    _launch(dev, lib.gocr_op_linear_ce, x.data_ptr(), w.data_ptr(), labels.data_ptr(), loss.data_ptr(), lse.data_ptr(),
            T, V, H, ws.data_ptr(), ws.numel())
    return loss, lse


def op_linear_ce_backward(dloss, x, w, labels, lse, workspace=None, loss=None):
    """(dx [T, H], dw [V, H]) bf16: the gradient of sum(dloss * loss) of
    op_linear_ce, from its lse; dloss fp32 [T] holds the rows' weights.  With
    the forward call's loss, too, the gradient of rows whose loss is small
    (below 1e-3) keeps its relative precision."""
    torch = _torch()
    lib = load()
    _lead("x", x, 2, torch.bfloat16)
    dev, (T, H), V = x.device, x.shape, w.shape[0]
    _want("x", x, (T, H), torch.bfloat16, dev)
    _want("w", w, (V, H), torch.bfloat16, dev)
    _want("labels", labels, (T,), torch.int32, dev)
    _want("dloss", dloss, (T,), torch.float32, dev)
    _want("lse", lse, (T,), torch.float32, dev)
    if loss is not None:
        _want("loss", loss, (T,), torch.float32, dev)
    _ready(dev, (T, V, H), dloss, x, w, lse, loss)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = _workspace(workspace, lib.gocr_op_linear_ce_backward_workspace(T, V, H), dev)
    _launch(dev, lib.gocr_op_linear_ce_backward_with_loss, dloss.data_ptr(), x.data_ptr(), w.data_ptr(), labels.data_ptr(),
            loss.data_ptr() if loss is not None else None, lse.data_ptr(), dx.data_ptr(), dw.data_ptr(), T, V, H, ws.data_ptr(), ws.numel())
    return dx, dw


# ----------------------------------------------------------------------------
# paged KV cache (serving: no gradients)
# ----------------------------------------------------------------------------

class PageStep(NamedTuple):
    """What op_page_step returns: int32 tensors on the device."""
    n_free: object   # [1] the stack's height after the step
    held: object     # [n_req] the next step's held
    kv_len: object   # [n_req] op_attention_paged's kv_len (0: refused)
    cu_rows: object  # [n_req + 1] request r's rows are cu_rows[r] .. cu_rows[r + 1] - 1
    pos: object      # [rows] position of each row, -1 of refused requests' and behind the last one
    slots: object    # [rows] its slot in the cache, or -1


def op_page_step(held, start, end, table, free_pages, n_free, page_size: int, rows: int) -> PageStep:
    """Block table, positions and slots of the next forward, from the requests'
    lengths (int32 [n_req] each, on the device): request r holds the pages of
    held[r] positions, its rows are positions start[r] .. end[r] - 1, and
    afterwards it holds the pages of end[r] positions, new ones taken from the
    stack free_pages [n_pages] (n_free [1] of them free) or those behind given
    back to it.  table [n_req, max_pages] and free_pages are updated in place;
    rows is the number of rows that the forward is laid out for.  A request
    whose pages do not fit is refused, and from the first one on whose rows do not
    fit all are, ends and rollbacks among them: a refused request keeps what it
    holds, as the returned held says."""
    torch = _torch()
    _lead("table", table, 2, torch.int32)
    dev, (R, width), n_pages = table.device, table.shape, free_pages.numel()
    _ints(dev, ("held", held, (R,)), ("start", start, (R,)), ("end", end, (R,)), ("table", table, (R, width)),
          ("free_pages", free_pages, (n_pages,)), ("n_free", n_free, (1,)))
    _ready(dev, (R, width, page_size, n_pages, rows))
    # (views that share no version counter: half the time of split)
    out = torch.unsafe_split_with_sizes(torch.empty((2 + 3 * R + 2 * rows,), dtype=torch.int32, device=dev),
                                        (1, R, R, R + 1, rows, rows))
    at = out[0].data_ptr()
    _launch(dev, load().gocr_op_page_step, held.data_ptr(), start.data_ptr(), end.data_ptr(), R, table.data_ptr(), width,
            page_size, free_pages.data_ptr(), n_pages, n_free.data_ptr(), at, at + 4, at + 4 * (1 + R),
            at + 4 * (1 + 2 * R), at + 4 * (2 + 3 * R), at + 4 * (2 + 3 * R + rows), rows)
    return PageStep(*out)


def _ints(device, *operands):
    """Check int32 operands, (name, tensor, shape) each, as _want does."""
    i32 = _torch().int32
    for name, t, shape in operands:
        if not (t.dtype is i32 and t.shape == shape and t.is_contiguous() and t.device == device):
            _want(name, t, shape, i32, device)


def _cache_args(q, k_cache, v_cache):
    """Check q [T, Hq, d] and a layer's pages, [n_pages, Hkv, page_size, d] each,
    in any order of the strides, all bf16; returns (PagedKV, device, T, Hq, Hkv, d, q's row pitch)."""
    bf16, dev, shape, pages = _torch().bfloat16, q.device, q.shape, k_cache.shape
    if len(shape) == 3 and len(pages) == 4 and v_cache.shape == pages and k_cache.dtype is v_cache.dtype is q.dtype is bf16:
        (T, Hq, d), (n, Hkv, ps, dk) = shape, pages
        qs, ks, vs = q.stride(), k_cache.stride(), v_cache.stride()
        if (dk == d and qs[2] == ks[3] == vs[3] == 1 and (Hq == 1 or qs[1] == d) and k_cache.device == dev
                and v_cache.device == dev and not (n | Hkv | ps) >> 31):
            kv = PagedKV(k_cache.data_ptr(), v_cache.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], n, ps, Hkv, d)
            return kv, dev, T, Hq, Hkv, d, qs[0] if T > 1 else Hq * d
    # what is wrong
    _lead("q", q, 3, bf16)
    _lead("k_cache", k_cache, 4, bf16)
    _lead("v_cache", v_cache, 4, bf16)
    if v_cache.shape != pages:
        raise ValueError(f"v_cache must be {list(pages)}, got {list(v_cache.shape)}")
    if k_cache.stride(3) != 1 or v_cache.stride(3) != 1:
        raise ValueError("the elements of a head must be contiguous in k_cache and v_cache")
    if k_cache.device != dev or v_cache.device != dev:
        raise ValueError(f"k_cache is on {k_cache.device}, v_cache on {v_cache.device}, q is on {dev}")
    if pages[3] != shape[2]:
        raise ValueError(f"the cache holds heads of {pages[3]}, q has heads of {shape[2]}")
    _rows("q", q, shape[0], None, shape[2], dev)
    raise ValueError(f"a size of {list(pages)} is outside 0 .. 2^31 - 1")


def op_kv_write_paged(q, k, v, pos, slots, k_cache, v_cache, theta: float = 10000.0, q_out=None):
    """Rotary embedding of q [T, Hq, d] and k [T, Hkv, d] at positions pos (int32
    [T]), and the write of k and v into slots (int32 [T], page * page_size +
    offset, distinct) of k_cache and v_cache [n_pages, Hkv, page_size, d] bf16
    (strides in any order).  Rows may be views of one fused projection.  Returns
    the rotated q [T, Hq, d], written into q_out when given; rows whose slot is
    outside the cache are skipped."""
    torch = _torch()
    kv, dev, T, Hq, Hkv, d, ldq = _cache_args(q, k_cache, v_cache)
    ldk, ldv = _rows("k", k, T, Hkv, d, dev), _rows("v", v, T, Hkv, d, dev)
    _ints(dev, ("pos", pos, (T,)), ("slots", slots, (T,)))
    _ready(dev, (T, Hq), q, k, v, k_cache, v_cache)
    if q_out is None:
        q_out = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=dev)
    else:
        _want("q_out", q_out, (T, Hq, d), torch.bfloat16, dev)
    _launch(dev, load().gocr_op_kv_write_paged, q.data_ptr(), k.data_ptr(), v.data_ptr(), pos.data_ptr(),
            slots.data_ptr(), q_out.data_ptr(), kv, T, Hq, ldq, ldk, ldv, theta)
    return q_out


def op_attention_paged(q, k_cache, v_cache, table, cu_rows, kv_len, kind: int = FWD_VERIFY, scale=None, workspace=None,
                       o=None, lse=None):
    """Attention of each request's new rows over its pages: q [T, Hq, d] bf16
    (rows may be views of one fused projection), k_cache and v_cache [n_pages,
    Hkv, page_size, d] bf16 (strides in any order), table int32 [n_req,
    max_pages], cu_rows int32 [n_req + 1] and kv_len int32 [n_req] (the new
    rows' keys counted) on the device, as op_page_step gives them.  Row i of a
    request's n is at position kv_len - n + i and reads the keys up to it;
    kind=FWD_DRAFT: the rows behind the first read all kv_len keys.  Returns (o
    [T, Hq, d] bf16, lse [Hq, T] fp32), written into o and lse when given; a row
    without keys gets 0 and -inf, rows of no request are not written.  The last
    bits of a row depend on the lengths of all requests of the call, so a verify
    window's row need not equal a single token's bit for bit: rounds of draft and
    verify over pages are not bit-identical to a loop of single tokens, as the
    decoder's are.  A non-finite v of a new row may reach rows before it of the
    same request."""
    torch = _torch()
    lib = load()
    kv, dev, T, Hq, Hkv, d, ldq = _cache_args(q, k_cache, v_cache)
    _lead("table", table, 2, torch.int32)
    R, width = table.shape
    _ints(dev, ("table", table, (R, width)), ("cu_rows", cu_rows, (R + 1,)), ("kv_len", kv_len, (R,)))
    _ready(dev, (R, width, T, Hq), q, k_cache, v_cache)
    if o is None:
        o = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=dev)
    else:
        _want("o", o, (T, Hq, d), torch.bfloat16, dev)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
    else:
        _want("lse", lse, (Hq, T), torch.float32, dev)
    need = lib.gocr_op_attention_paged_workspace(T, Hq, Hkv, d)
    ws = _workspace(workspace, need, dev)
    _launch(dev, lib.gocr_op_attention_paged, q.data_ptr(), kv, table.data_ptr(), width, cu_rows.data_ptr(),
            kv_len.data_ptr(), kind, o.data_ptr(), lse.data_ptr(), R, T, Hq, ldq, d ** -0.5 if scale is None else scale,
            ws.data_ptr(), need if workspace is None else ws.numel())
    return o, lse


def op_status(device="cuda") -> None:
    """Wait for the device's current stream; raise when a kernel of these
    operators gave up a wait since this thread last asked.  The other calls do
    not wait and do not ask: a program does, once a step or before it trusts
    what it saves."""
    torch = _torch()
    with torch.cuda.device(device):
        _check(load().gocr_op_status(torch.cuda.current_stream().cuda_stream))
