"""ctypes binding of libsdv (``include/sdv.h``), torch tensors in and out.

Argument marshalling only: every step of the verification runs in the CUDA
kernels of ``libsdv.so``.  There is no fallback: if the library is missing or
does not load, every call raises.

The functions keep the C names (``sdv_create``, ``sdv_verify``,
``sdv_verify_ex``, ``sdv_verify_host``, ``sdv_sync``, ``sdv_last_error``,
``sdv_destroy``, ``sdv_plan``); ``Verifier`` wraps a context.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsdv.so")

SDV_OK, SDV_ERR_ARG, SDV_ERR_CUDA, SDV_ERR_OOM, SDV_ERR_DEVICE_DATA, SDV_ERR_SCRATCH = 0, 1, 2, 3, 4, 5
SDV_BF16, SDV_F32, SDV_F16, SDV_E4M3 = 0, 1, 2, 3
SDV_FLAG_SHARED_Q = 1
SDV_FLAG_GREEDY = 2
SDV_FLAG_SHARED_PREFIX_ROW = 4
STATUS_NAMES = {0: "SDV_OK", 1: "SDV_ERR_ARG", 2: "SDV_ERR_CUDA", 3: "SDV_ERR_OOM",
                4: "SDV_ERR_DEVICE_DATA", 5: "SDV_ERR_SCRATCH"}
STATIC_SCRATCH_BYTES = 8 << 20
SDV_STATUS_BAD_TOKEN, SDV_STATUS_TIMEOUT = 1, 8
SDV_STATUS_BAD_ROW, SDV_STATUS_BAD_PARAM = 2, 4
SDV_STATUS_BAD_LENGTH = 16
SDV_STATUS_BAD_PAGE = 64
SDV_STATUS_NO_PAGES = 128
SDV_ROPE_PLAIN, SDV_ROPE_LINEAR, SDV_ROPE_BASE, SDV_ROPE_PARTS = 0, 1, 2, 3
SDV_HOOK_SAMPLE_NO_COPY = 1
SDV_HOOK_ATTN_NO_COPY = 2

# Every entry point of include/sdv.h, with its ctypes signature.
_VP, _I, _I64, _U64, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float


class _KVCache(ctypes.Structure):
    """sdv_kv_cache of include/sdv.h."""
    _fields_ = [("k", _VP), ("v", _VP), ("k_exp", _VP), ("v_exp", _VP), ("page_stride", _I64),
                ("exp_page_stride", _I64), ("pages", _I), ("page_size", _I), ("kv_heads", _I),
                ("head_dim", _I), ("dtype", _I)]


_KVP = ctypes.POINTER(_KVCache)
SIGNATURES = {
    "sdv_create": (_I, [ctypes.POINTER(_VP), _I, _I, _I, _I, _I, _VP]),
    "sdv_create_ex": (_I, [ctypes.POINTER(_VP), _I, _I, _I, _I, _I, _VP, ctypes.c_uint]),
    "sdv_verify": (_I, [_VP, _VP, _VP, _VP, _F, _U64, _VP, _VP, _VP]),
    "sdv_verify_ex": (_I, [_VP, _VP, _VP, _VP, _F, _VP, _U64, _VP, _VP, _VP, _VP, _VP]),
    "sdv_verify_len": (_I, [_VP, _VP, _VP, _VP, _VP, _F, _VP, _U64, _VP, _VP, _VP, _VP, _VP]),
    "sdv_verify_qstat": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _F, _VP, _U64, _VP, _VP, _VP, _VP,
                              _VP]),
    "sdv_verify_host": (_I, [_VP, _VP, _VP, _VP, _F, _VP, _U64, _VP, _VP, _VP]),
    "sdv_sync": (_I, [_VP]),
    "sdv_last_error": (ctypes.c_char_p, [_VP]),
    "sdv_destroy": (None, [_VP]),
    "sdv_plan": (_I, [_VP, ctypes.POINTER(_I), ctypes.POINTER(_I64), ctypes.POINTER(_I),
                      ctypes.POINTER(_I)]),
    "sdv_set_stream": (_I, [_VP, _VP]),
    "sdv_set_test_hooks": (_I, [_VP, ctypes.c_uint]),
    "sdv_profile_enable": (_I, [_VP, _I]),
    "sdv_profile_read": (_I, [_VP, ctypes.POINTER(_F), ctypes.POINTER(_I)]),
    "sdv_verify_static": (_I, [_I, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _F, _VP, _U64, _VP, _VP, _VP]),
    "sdv_cps": (_I, [_I, _I, _I, _I, _VP, _VP, _F, _VP, _F, _I, _I, _I, _VP, _VP, _VP, _VP, _VP,
                     _VP, _VP, _VP]),
    "sdv_cps_ex": (_I, [_I, _I, _I, _I, _VP, _VP, _F, _VP, _F, _I, _I, _I, _VP, _VP, _VP, _VP,
                        _VP, _VP, _VP, _VP, _VP]),
    "sdv_cps_prune": (_I, [_I, _I, _I, _I, _VP, _VP, _F, _VP, _F, _I, _VP, _VP, _VP, _VP]),
    "sdv_cps_beam": (_I, [_I, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "sdv_adl_state_words": (_I, [_I]),
    "sdv_adl_step_host": (_I, [_I, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP]),
    "sdv_adl_step": (_I, [_I, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP]),
    "sdv_tree_build": (_I, [_I, _I, _I] + [_VP] * 11),
    "sdv_rope_freqs": (_I, [_I, ctypes.c_double, _I, ctypes.c_double, ctypes.c_double,
                            ctypes.c_double, ctypes.c_double, _VP, _VP]),
    "sdv_rope": (_I, [_I64, _I, _I, _I, _I, _I, _I, _VP, _VP, _I64, _I64, _VP, _I64, _I64, _VP, _VP,
                      _F, _VP, _I64, _I64, _VP, _I64, _I64]),
    "sdv_kv_write": (_I, [_KVP, _I, _I, _I, _VP, _VP, _I64, _I64, _I64, _VP, _I64, _I64, _I64, _VP,
                          _I, _VP, _VP, _VP]),
    "sdv_kv_read": (_I, [_KVP, _I, _I, _I, _VP, _VP, _VP, _VP, _I, _VP, _VP, _VP]),
    "sdv_kv_commit": (_I, [_KVP, _I, _I, _I, _VP, _VP, _I, _VP, _VP, _VP, _VP, _VP, _VP]),
    "sdv_tree_attn_workspace": (ctypes.c_size_t, []),
    "sdv_tree_attn": (_I, [_KVP, _I, _I, _I, _I, _VP, _VP, _I64, _I64, _I64, _VP, _I, _VP, _VP, _VP,
                           _I64, _F, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "sdv_prefix_attn_workspace": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "sdv_prefix_attn": (_I, [_KVP, _I, _I, _I, _I, _I, _VP, _VP, _I64, _I64, _I64, _VP, _I, _VP, _VP, _I,
                             _VP, _VP, _VP, _I64, _F, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "sdv_set_attn_test_hooks": (_I, [ctypes.c_uint]),
    "sdv_logits_process": (_I, [_I, _I, _I, _I, _I, _VP, _VP, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                _I, _VP, _VP, _VP, _VP, _VP]),
    "sdv_counts_commit": (_I, [_I, _I, _I, _I] + [_VP] * 7),
    "sdv_pages_extend": (_I, [_I] * 5 + [_VP] * 12),
    "sdv_pages_release": (_I, [_I] * 4 + [_VP] * 7),
    "sdv_sample": (_I, [_I64, _I, _I, _I, _VP, _VP, _I64] + [_VP] * 9),
    "sdv_logits_truncate": (_I, [_I64, _I, _I, _I, _VP, _VP, _I64, _VP, _VP, _VP, _VP, _VP, _I64, _VP,
                                 _VP]),
}

_lib = None


class SdvError(RuntimeError):
    def __init__(self, status: int, msg: str = ""):
        super().__init__("%s%s" % (STATUS_NAMES.get(status, str(status)), (": " + msg) if msg else ""))
        self.status = status


def load(build: bool = False) -> ctypes.CDLL:
    """Load libsdv.so (optionally building it first).  Raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if build:
        from . import build as _b
        _b.build()
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libsdv.so is not built (run draft_verification_sdv_gb300.build.build());"
                           " there is no CPU fallback")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _dev_ptr(t: Optional[torch.Tensor], dtype=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return ctypes.c_void_p(t.data_ptr())


def _per_seq(t: Optional[torch.Tensor], B: int, name: str) -> None:
    """A per-sequence array must hold one entry per sequence: the library
    reads B of them."""
    if t is not None and t.numel() != B:
        raise ValueError("%s must have one entry per sequence (%d)" % (name, B))


def _host_ptr(t: Optional[torch.Tensor], dtype=None, name="tensor"):
    if t is None:
        return None
    if t.is_cuda:
        raise ValueError("%s must be a host tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return ctypes.c_void_p(t.data_ptr())


def _dtype_code(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return SDV_BF16
    if dtype == torch.float32:
        return SDV_F32
    raise TypeError("logits must be bfloat16 or float32")


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def sdv_create(B: int, K: int, gamma: int, V: int, dtype: torch.dtype = torch.bfloat16,
               stream=None, flags: int = 0) -> ctypes.c_void_p:
    ctx = ctypes.c_void_p()
    st = load().sdv_create_ex(ctypes.byref(ctx), B, K, gamma, V, _dtype_code(dtype),
                              ctypes.c_void_p(_stream_handle(stream)), int(flags))
    if st != SDV_OK:
        raise SdvError(st, "sdv_create(B=%d, K=%d, gamma=%d, V=%d)" % (B, K, gamma, V))
    return ctx


def sdv_verify(ctx, p_logits, q_logits, drafts, temperature, seed, out_sel, out_accept_len,
               out_next_token) -> int:
    return load().sdv_verify(ctx, _dev_ptr(p_logits, name="p_logits"),
                             _dev_ptr(q_logits, name="q_logits"),
                             _dev_ptr(drafts, torch.int32, "drafts"), float(temperature),
                             int(seed) & 0xFFFFFFFFFFFFFFFF, _dev_ptr(out_sel, torch.int32, "out_sel"),
                             _dev_ptr(out_accept_len, torch.int32, "out_accept_len"),
                             _dev_ptr(out_next_token, torch.int32, "out_next_token"))


def sdv_verify_ex(ctx, p_logits, q_logits, drafts, temperature, temperature_per_seq, seed,
                  out_sel, out_accept_len, out_next_token, out_scores=None, out_lse=None) -> int:
    return load().sdv_verify_ex(
        ctx, _dev_ptr(p_logits, name="p_logits"), _dev_ptr(q_logits, name="q_logits"),
        _dev_ptr(drafts, torch.int32, "drafts"), float(temperature),
        _dev_ptr(temperature_per_seq, torch.float32, "temperature_per_seq"),
        int(seed) & 0xFFFFFFFFFFFFFFFF, _dev_ptr(out_sel, torch.int32, "out_sel"),
        _dev_ptr(out_accept_len, torch.int32, "out_accept_len"),
        _dev_ptr(out_next_token, torch.int32, "out_next_token"),
        _dev_ptr(out_scores, torch.float32, "out_scores"),
        _dev_ptr(out_lse, torch.float32, "out_lse"))


def sdv_verify_qstat(ctx, p_logits, q_logits, drafts, draft_len, q_row_stat, temperature,
                     temperature_per_seq, seed, out_sel, out_accept_len, out_next_token,
                     out_scores=None, out_lse=None) -> int:
    return load().sdv_verify_qstat(
        ctx, _dev_ptr(p_logits, name="p_logits"), _dev_ptr(q_logits, name="q_logits"),
        _dev_ptr(drafts, torch.int32, "drafts"), _dev_ptr(draft_len, torch.int32, "draft_len"),
        _dev_ptr(q_row_stat, torch.float32, "q_row_stat"), float(temperature),
        _dev_ptr(temperature_per_seq, torch.float32, "temperature_per_seq"),
        int(seed) & 0xFFFFFFFFFFFFFFFF, _dev_ptr(out_sel, torch.int32, "out_sel"),
        _dev_ptr(out_accept_len, torch.int32, "out_accept_len"),
        _dev_ptr(out_next_token, torch.int32, "out_next_token"),
        _dev_ptr(out_scores, torch.float32, "out_scores"),
        _dev_ptr(out_lse, torch.float32, "out_lse"))


def sdv_verify_len(ctx, p_logits, q_logits, drafts, draft_len, temperature, temperature_per_seq,
                   seed, out_sel, out_accept_len, out_next_token, out_scores=None,
                   out_lse=None) -> int:
    return load().sdv_verify_len(
        ctx, _dev_ptr(p_logits, name="p_logits"), _dev_ptr(q_logits, name="q_logits"),
        _dev_ptr(drafts, torch.int32, "drafts"), _dev_ptr(draft_len, torch.int32, "draft_len"),
        float(temperature), _dev_ptr(temperature_per_seq, torch.float32, "temperature_per_seq"),
        int(seed) & 0xFFFFFFFFFFFFFFFF, _dev_ptr(out_sel, torch.int32, "out_sel"),
        _dev_ptr(out_accept_len, torch.int32, "out_accept_len"),
        _dev_ptr(out_next_token, torch.int32, "out_next_token"),
        _dev_ptr(out_scores, torch.float32, "out_scores"),
        _dev_ptr(out_lse, torch.float32, "out_lse"))


def sdv_verify_host(ctx, p_logits, q_logits, drafts, temperature, temperature_per_seq, seed,
                    out_sel, out_accept_len, out_next_token) -> int:
    return load().sdv_verify_host(
        ctx, _host_ptr(p_logits, name="p_logits"), _host_ptr(q_logits, name="q_logits"),
        _host_ptr(drafts, torch.int32, "drafts"), float(temperature),
        _host_ptr(temperature_per_seq, torch.float32, "temperature_per_seq"),
        int(seed) & 0xFFFFFFFFFFFFFFFF, _host_ptr(out_sel, torch.int32, "out_sel"),
        _host_ptr(out_accept_len, torch.int32, "out_accept_len"),
        _host_ptr(out_next_token, torch.int32, "out_next_token"))


def sdv_sync(ctx) -> int:
    return load().sdv_sync(ctx)


def sdv_last_error(ctx) -> str:
    r = load().sdv_last_error(ctx)
    return r.decode() if r else ""


def sdv_destroy(ctx) -> None:
    load().sdv_destroy(ctx)


def sdv_plan(ctx) -> dict:
    g, ck, cv, cl = _I(), _I(), _I64(), _I()
    st = load().sdv_plan(ctx, ctypes.byref(g), ctypes.byref(cv), ctypes.byref(ck), ctypes.byref(cl))
    if st != SDV_OK:
        raise SdvError(st)
    return {"rowpass_ctas": g.value, "chunk_vectors": cv.value, "chunks_per_row": ck.value,
            "sample_cluster": cl.value}


def sdv_profile_enable(ctx, enable: bool = True) -> int:
    return load().sdv_profile_enable(ctx, 1 if enable else 0)


def sdv_profile_read(ctx):
    """(mean ms of [row pass, select, sample], number of steps); clears the record."""
    ms = (_F * 3)()
    n = _I()
    st = load().sdv_profile_read(ctx, ms, ctypes.byref(n))
    if st != SDV_OK:
        raise SdvError(st, sdv_last_error(ctx))
    return [float(x) for x in ms], n.value


def sdv_verify_static(B, K, gamma, V, dtype, stream, p_logits, q_logits, drafts, temperature,
                      temperature_per_seq, seed, out_sel, out_accept_len, out_next_token) -> int:
    """Allocation-free step (no context): scratch lives in a static device array."""
    return load().sdv_verify_static(
        B, K, gamma, V, _dtype_code(dtype), ctypes.c_void_p(_stream_handle(stream)),
        _dev_ptr(p_logits, name="p_logits"), _dev_ptr(q_logits, name="q_logits"),
        _dev_ptr(drafts, torch.int32, "drafts"), float(temperature),
        _dev_ptr(temperature_per_seq, torch.float32, "temperature_per_seq"),
        int(seed) & 0xFFFFFFFFFFFFFFFF, _dev_ptr(out_sel, torch.int32, "out_sel"),
        _dev_ptr(out_accept_len, torch.int32, "out_accept_len"),
        _dev_ptr(out_next_token, torch.int32, "out_next_token"))


def sdv_cps(q_marginals, tau: float = 0.8, mmax: int = 15, beam: int = 3, eos_id: int = -1,
            temperature: float = 1.0, temps: Optional[torch.Tensor] = None, stream=None,
            out: Optional[dict] = None, row_stat: bool = False) -> dict:
    """Causal-consistency path search over drafter marginals q [B, gamma, V]
    (candidate pruning by cumulative mass, EOS cut, beam by drafter
    confidence).  Enqueues on `stream` (default: the current stream) and
    returns the output tensors; `out` (a dict this returned for the same
    shapes) reuses them.  With `row_stat`, out["row_stat"] [B, gamma, 4] holds
    each marginal row's softmax statistics (sdv_cps_ex), which a Verifier call
    takes as `q_stat` so that it does not stream the marginals again."""
    B, G, V = q_marginals.shape
    _per_seq(temps, B, "temps")
    dev = q_marginals.device
    if out is not None and row_stat and "row_stat" not in out:
        out["row_stat"] = torch.empty((B, G, 4), dtype=torch.float32, device=dev)
    out = out if out is not None else {
        "cand_ids": torch.empty((B, G, mmax), dtype=torch.int32, device=dev),
        "cand_logp": torch.empty((B, G, mmax), dtype=torch.float32, device=dev),
        "cand_logit": torch.empty((B, G, mmax), dtype=torch.float32, device=dev),
        "ncand": torch.empty((B, G), dtype=torch.int32, device=dev),
        "paths": torch.empty((B, beam, G), dtype=torch.int32, device=dev),
        "path_logp": torch.empty((B, beam), dtype=torch.float32, device=dev),
        "npaths": torch.empty((B,), dtype=torch.int32, device=dev),
        "lat_len": torch.empty((B,), dtype=torch.int32, device=dev),
    }
    if row_stat and "row_stat" not in out:
        out["row_stat"] = torch.empty((B, G, 4), dtype=torch.float32, device=dev)
    st = load().sdv_cps_ex(B, G, V, _dtype_code(q_marginals.dtype),
                           ctypes.c_void_p(_stream_handle(stream)),
                           _dev_ptr(q_marginals, name="q_marginals"), float(temperature),
                           _dev_ptr(temps, torch.float32, "temps"), float(tau), int(mmax), int(beam),
                           int(eos_id), *[_dev_ptr(out[k]) for k in ("cand_ids", "cand_logp",
                                                                     "cand_logit", "ncand", "paths",
                                                                     "path_logp", "npaths",
                                                                     "lat_len")],
                           _dev_ptr(out["row_stat"], torch.float32, "row_stat") if row_stat else None)
    if st != SDV_OK:
        raise SdvError(st, "sdv_cps")
    return out


def _cps_lattice(B, G, mmax, dev):
    return {"cand_ids": torch.empty((B, G, mmax), dtype=torch.int32, device=dev),
            "cand_logp": torch.empty((B, G, mmax), dtype=torch.float32, device=dev),
            "cand_logit": torch.empty((B, G, mmax), dtype=torch.float32, device=dev),
            "ncand": torch.empty((B, G), dtype=torch.int32, device=dev)}


def sdv_cps_prune(q_marginals, tau: float = 0.8, mmax: int = 15, temperature: float = 1.0,
                  temps: Optional[torch.Tensor] = None, stream=None, out: Optional[dict] = None) -> dict:
    """The pruning half of sdv_cps: every row's candidate list (no EOS cut).
    `out` (the dict this returns) may be passed back to reuse its tensors."""
    B, G, V = q_marginals.shape
    _per_seq(temps, B, "temps")
    out = out if out is not None else _cps_lattice(B, G, mmax, q_marginals.device)
    st = load().sdv_cps_prune(B, G, V, _dtype_code(q_marginals.dtype),
                              ctypes.c_void_p(_stream_handle(stream)),
                              _dev_ptr(q_marginals, name="q_marginals"), float(temperature),
                              _dev_ptr(temps, torch.float32, "temps"), float(tau), int(mmax),
                              *[_dev_ptr(out[k]) for k in ("cand_ids", "cand_logp", "cand_logit",
                                                           "ncand")])
    if st != SDV_OK:
        raise SdvError(st, "sdv_cps_prune")
    return out


def sdv_cps_beam(lattice: dict, V: int, beam: int = 3, eos_id: int = -1, stream=None,
                 out: Optional[dict] = None) -> dict:
    """The beam half of sdv_cps over a lattice from sdv_cps_prune (trimmed in
    place at an EOS end).  Returns the lattice dict with the path tensors;
    `out` (a dict this returned for the same shapes) reuses them."""
    B, G, mmax = lattice["cand_ids"].shape
    dev = lattice["cand_ids"].device
    if out is None:
        out = dict(lattice)
        out.update({"paths": torch.empty((B, beam, G), dtype=torch.int32, device=dev),
                    "path_logp": torch.empty((B, beam), dtype=torch.float32, device=dev),
                    "npaths": torch.empty((B,), dtype=torch.int32, device=dev),
                    "lat_len": torch.empty((B,), dtype=torch.int32, device=dev)})
    else:
        out.update(lattice)
    st = load().sdv_cps_beam(B, G, int(V), int(mmax), int(beam), int(eos_id),
                             ctypes.c_void_p(_stream_handle(stream)),
                             *[_dev_ptr(out[k]) for k in ("cand_ids", "cand_logp", "cand_logit",
                                                          "ncand", "paths",
                                                          "path_logp", "npaths", "lat_len")])
    if st != SDV_OK:
        raise SdvError(st, "sdv_cps_beam")
    return out


class DraftLengthController:
    """Adaptive draft length for B sequences (the library's rule; see
    sdv_adl_step in include/sdv.h).  On a CUDA device the state, the lengths
    and the update stay on the device (`step` enqueues one kernel); on the
    host the same rule runs in the library's C code."""

    def __init__(self, B: int, k0, window: int = 1, kmin: int = 1, kmax: int = 64, up: int = 2,
                 down: int = 1, device="cuda"):
        words = load().sdv_adl_state_words(int(window))
        if words < 0:
            raise SdvError(SDV_ERR_ARG, "window")
        self.B, self.window, self.kmin, self.kmax, self.up, self.down = B, window, kmin, kmax, up, down
        self.device = torch.device(device)
        self.state = torch.zeros((B, words), dtype=torch.int32, device=self.device)
        self.k = torch.as_tensor(k0, dtype=torch.int32).expand(B).clone().to(self.device)
        self.status = (torch.zeros(1, dtype=torch.int32, device=self.device)
                       if self.device.type == "cuda" else None)

    def step(self, gen_len: torch.Tensor, acc_len: torch.Tensor, stream=None) -> torch.Tensor:
        """Record one step's generated and accepted lengths [B] (int32, on the
        controller's device) and return the next draft lengths (self.k)."""
        _per_seq(gen_len, self.B, "gen_len")
        _per_seq(acc_len, self.B, "acc_len")
        g = gen_len.to(torch.int32).contiguous()
        a = acc_len.to(torch.int32).contiguous()
        if self.device.type == "cuda":
            st = load().sdv_adl_step(self.B, self.window, self.kmin, self.kmax, self.up, self.down,
                                     ctypes.c_void_p(_stream_handle(stream)), _dev_ptr(g), _dev_ptr(a),
                                     _dev_ptr(self.k), _dev_ptr(self.state), _dev_ptr(self.status))
        else:
            st = load().sdv_adl_step_host(self.B, self.window, self.kmin, self.kmax, self.up,
                                          self.down, _host_ptr(g), _host_ptr(a), _host_ptr(self.k),
                                          _host_ptr(self.state))
        if st != SDV_OK:
            raise SdvError(st, "sdv_adl_step")
        return self.k


def sdv_set_stream(ctx, stream) -> int:
    return load().sdv_set_stream(ctx, ctypes.c_void_p(_stream_handle(stream)))


def sdv_set_test_hooks(ctx, hooks: int) -> int:
    """Fault-path test hooks of a context (SDV_HOOK_* bits; 0 = none)."""
    return load().sdv_set_test_hooks(ctx, int(hooks))


class Verifier:
    """One context for batches of shape (B, K, gamma, V).

    ``v(p, q, drafts, ...)`` enqueues a step on the context's stream and returns
    the output tensors; ``v.sync()`` waits and raises on a device-side error.
    """

    def __init__(self, B: int, K: int, gamma: int, V: int, dtype=torch.bfloat16,
                 device=None, stream=None, shared_q: bool = False, greedy: bool = False,
                 shared_prefix_row: bool = False):
        self.B, self.K, self.gamma, self.V, self.dtype = B, K, gamma, V, dtype
        self.shared_q = shared_q
        self.greedy = greedy
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        with torch.cuda.device(self.device):
            self.stream = stream
            self.ctx = sdv_create(B, K, gamma, V, dtype, stream,
                                  (SDV_FLAG_SHARED_Q if shared_q else 0) |
                                  (SDV_FLAG_GREEDY if greedy else 0) |
                                  (SDV_FLAG_SHARED_PREFIX_ROW if shared_prefix_row else 0))

    def __call__(self, p_logits, q_logits, drafts, temperature: float = 1.0, seed: int = 0,
                 temps: Optional[torch.Tensor] = None, scores: bool = False, lse: bool = False,
                 out: Optional[dict] = None, draft_len: Optional[torch.Tensor] = None,
                 q_stat: Optional[torch.Tensor] = None) -> dict:
        """One verification step; `draft_len` (int32 [B] on the device) gives
        each sequence's draft length (sdv_verify_len), else all are gamma;
        `q_stat` (float32 [rows_q, 4], e.g. sdv_cps(..., row_stat=True)
        ["row_stat"]) supplies the drafter rows' softmax statistics, so the
        q rows are not streamed (sdv_verify_qstat)."""
        B, K, G, V = self.B, self.K, self.gamma, self.V
        q_shape = (B, G, V) if self.shared_q else (B, K, G, V)
        if tuple(p_logits.shape) != (B, K, G + 1, V):
            raise ValueError("p_logits must be [B,K,gamma+1,V]")
        if not self.greedy and (q_logits is None or tuple(q_logits.shape) != q_shape):
            raise ValueError("q_logits must be %s" % (list(q_shape),))
        if tuple(drafts.shape) != (B, K, G):
            raise ValueError("drafts must be [B,K,gamma]")
        if p_logits.dtype != self.dtype or (q_logits is not None and q_logits.dtype != self.dtype):
            raise TypeError("logits must be %s" % self.dtype)
        _per_seq(temps, B, "temps")
        _per_seq(draft_len, B, "draft_len")
        dev = p_logits.device
        if out is None:
            out = {
                "sel": torch.empty(B, dtype=torch.int32, device=dev),
                "accept_len": torch.empty(B, dtype=torch.int32, device=dev),
                "next_token": torch.empty(B, dtype=torch.int32, device=dev),
            }
            if scores:
                out["scores"] = torch.empty((B, K), dtype=torch.float32, device=dev)
            if lse:
                out["lse"] = torch.empty((B, K, G + 1 if self.greedy else 2 * G + 1),
                                         dtype=torch.float32, device=dev)
        if q_stat is not None:
            rows_q = B * G if self.shared_q else B * K * G
            if not self.greedy and (q_stat.dtype != torch.float32 or q_stat.numel() != rows_q * 4):
                raise ValueError("q_stat must be float32 with %d x 4 entries (one per q row)"
                                 % rows_q)
            st = sdv_verify_qstat(self.ctx, p_logits, q_logits, drafts, draft_len, q_stat,
                                  temperature, temps, seed, out["sel"], out["accept_len"],
                                  out["next_token"], out.get("scores"), out.get("lse"))
        elif draft_len is None:
            st = sdv_verify_ex(self.ctx, p_logits, q_logits, drafts, temperature, temps, seed,
                               out["sel"], out["accept_len"], out["next_token"], out.get("scores"),
                               out.get("lse"))
        else:
            st = sdv_verify_len(self.ctx, p_logits, q_logits, drafts, draft_len, temperature, temps,
                                seed, out["sel"], out["accept_len"], out["next_token"],
                                out.get("scores"), out.get("lse"))
        if st != SDV_OK:
            raise SdvError(st, sdv_last_error(self.ctx))
        return out

    def set_stream(self, stream) -> None:
        """Enqueue later steps on `stream` (for CUDA-graph capture: the
        capturing stream).  The caller orders it after earlier steps."""
        st = sdv_set_stream(self.ctx, stream)
        if st != SDV_OK:
            raise SdvError(st, sdv_last_error(self.ctx))
        self.stream = stream

    def sync(self) -> None:
        st = sdv_sync(self.ctx)
        if st != SDV_OK:
            raise SdvError(st, sdv_last_error(self.ctx))

    def plan(self) -> dict:
        return sdv_plan(self.ctx)

    def close(self) -> None:
        if getattr(self, "ctx", None) is not None:
            sdv_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --------------------------------------------------------------------------
# The verifier's layer: draft tree, rotary positions, paged cache, attention
# of the tree over the cache, sampling parameters.
#
# These run once per layer and step, so the checks here read what torch holds
# and build no intermediate objects; whether a pointer is on the device is
# checked by the library.  With a `stream` of its own a call is ordered there: the
# caller orders what it reads before it and what reads its outputs after it.
# --------------------------------------------------------------------------

_HALF_TYPES = {torch.bfloat16: SDV_BF16, torch.float16: SDV_F16}
_CELL_TYPES = {torch.bfloat16: SDV_BF16, torch.float16: SDV_F16, torch.float8_e4m3fn: SDV_E4M3}
_ROPE_TYPES = {torch.bfloat16: SDV_BF16, torch.float16: SDV_F16, torch.float32: SDV_F32}


def _array(t: Optional[torch.Tensor], n: int, dtype: torch.dtype, name: str) -> Optional[int]:
    """Address of a contiguous device array of n entries (None stays None)."""
    if t is None:
        return None
    if t.dtype is dtype and t.is_cuda and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be contiguous with %d entries, got %s" % (name, n, tuple(t.shape)))
    return t.data_ptr()


def _rows_of(t: torch.Tensor, dims: int, name: str):
    """(shape, strides) of a device tensor whose innermost dimension is contiguous."""
    shape, stride = t.shape, t.stride()
    if len(stride) != dims:
        raise ValueError("%s must have %d dimensions, got %s" % (name, dims, tuple(shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if stride[-1] != 1 and shape[-1] != 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)
    return shape, stride


def _stream_of(t: torch.Tensor, stream) -> int:
    """Handle of `stream`, or of the current stream of t's device (asked for
    without building a Stream object: these calls come once per layer)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.device.index)
    return _stream_handle(stream)


def _empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """torch.empty for a call on `stream` (None: the current one).  Memory comes
    from the pool of the stream that writes it: a block of the current stream's
    may still be in use there.  And it goes back only when the current stream,
    where the caller reads it, is done with it too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device) if int(stream) else \
            torch.cuda.default_stream(device)
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if stream != here:
        t.record_stream(here)
    return t


def _type_of(types: dict, dtype: torch.dtype, name: str) -> int:
    code = types.get(dtype)
    if code is None:
        raise TypeError("%s must be one of %s, got %s" % (name, [str(t) for t in types], dtype))
    return code


def _page_stride(shape, stride) -> Optional[int]:
    """Elements from one page to the next (None: a page is not contiguous).  The
    stride of a dimension of one entry means nothing."""
    whole = 1
    for n, s in zip(shape[:0:-1], stride[:0:-1]):
        if n != 1 and s != whole:
            return None
        whole *= n
    return stride[0] if shape[0] != 1 else whole


def _cache_of(k_cache, v_cache, k_exp, v_exp) -> _KVCache:
    shape, ks = _rows_of(k_cache, 4, "k_cache")
    pages, heads, place, dim = shape
    dtype = k_cache.dtype
    code = _type_of(_CELL_TYPES, dtype, "the cache")
    vs = v_cache.stride()
    if pages > 1 and vs == ks and ks[1] == place * dim and ks[2] == dim:
        page = ks[0]
    else:
        page = _page_stride(shape, ks)
        if page != _page_stride(shape, vs):
            page = None
    if v_cache.shape != shape or v_cache.dtype != dtype or not v_cache.is_cuda or page is None:
        raise ValueError("k_cache and v_cache must be [pages, kv_heads, page_size, head_dim] of one "
                         "type and page stride, each page contiguous")
    exp_stride, ke, ve = 0, None, None
    if code == SDV_E4M3:
        if k_exp is None or v_exp is None:
            raise ValueError("an e4m3 cache needs k_exp and v_exp")
        for t, name in ((k_exp, "k_exp"), (v_exp, "v_exp")):
            eshape, es = _rows_of(t, 3, name)
            exp_stride = es[0] if pages > 1 and es[1] == place else _page_stride(eshape, es)
            if t.dtype != torch.uint8 or eshape != shape[:3] or exp_stride is None:
                raise ValueError("%s must be uint8 [pages, kv_heads, page_size], each page contiguous"
                                 % name)
        if k_exp.stride(0) != es[0] and _page_stride(shape[:3], k_exp.stride()) != exp_stride:
            raise ValueError("k_exp and v_exp must have one page stride")
        ke, ve = k_exp.data_ptr(), v_exp.data_ptr()
    elif k_exp is not None or v_exp is not None:
        raise ValueError("k_exp and v_exp belong to an e4m3 cache")
    return _KVCache(k_cache.data_ptr(), v_cache.data_ptr(), ke, ve, page, exp_stride, pages, place,
                    heads, dim, code)


def _table_of(block_table: torch.Tensor, B: int) -> int:
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != B:
        raise ValueError("block_table must be [%d, max_pages], got %s" % (B, tuple(shape)))
    return _array(block_table, block_table.numel(), torch.int32, "block_table")


def _status_of(status: Optional[torch.Tensor]) -> Optional[int]:
    return _array(status, 1, torch.int32, "status")


def sdv_tree_build(root: torch.Tensor, drafts: torch.Tensor,
                   draft_len: Optional[torch.Tensor] = None, stream=None,
                   out: Optional[dict] = None, status: Optional[torch.Tensor] = None) -> dict:
    """The tree of K drafts [B, K, gamma] behind each sequence's last token
    root [B] (all int32): its tokens, depths, ancestor mask, the drafts' nodes,
    the node of each verifier row, and the number of nodes.  `out` (a dict this
    returned for the same shapes) reuses the tensors."""
    B, K, G = drafts.shape
    N = 1 + K * G
    W = (N + 31) // 32
    shapes = {"tokens": (B, N), "depth": (B, N), "mask": (B, N, W), "nodes": (B, K, G),
              "rows": (B, K, G + 1), "count": (B,)}
    if out is None:
        out = {n: _empty(s, torch.int32, drafts.device, stream) for n, s in shapes.items()}
    at = []
    for n, s in shapes.items():
        size = 1
        for x in s:
            size *= x
        at.append(_array(out[n], size, torch.int32, n))
    st = load().sdv_tree_build(B, K, G, _stream_handle(stream), _array(root, B, torch.int32, "root"),
                               _array(drafts, B * K * G, torch.int32, "drafts"),
                               _array(draft_len, B, torch.int32, "draft_len"), *at,
                               _status_of(status))
    if st != SDV_OK:
        raise SdvError(st, "sdv_tree_build")
    return out


def sdv_rope_freqs(R: int, base: float = 10000.0, scaling: int = SDV_ROPE_PLAIN, factor: float = 1.0,
                   original: float = 8192, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """(rotary frequencies [R / 2] float32 on `device`, attention factor),
    scaled for long contexts by one of SDV_ROPE_*."""
    if R < 2:
        raise ValueError("R must be at least 2")
    f = torch.empty(R // 2, dtype=torch.float32)
    at = _F()
    st = load().sdv_rope_freqs(int(R), float(base), int(scaling), float(factor), float(original),
                               float(fast), float(slow), f.data_ptr(), ctypes.addressof(at))
    if st != SDV_OK:
        raise SdvError(st, "sdv_rope_freqs")
    return f.to(device), at.value


def sdv_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor,
             inv_freq: torch.Tensor, factor: float = 1.0, interleaved: bool = False,
             out_q: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None,
             stream=None):
    """Rotary positions of q [T, Hq, D] and k [T, Hk, D] (or None) at
    positions [T] int32: the first 2 * len(inv_freq) elements of each head turn.
    q and k may be strided views; out_q=q, out_k=k works in place.  Returns
    (out_q, out_k)."""
    (T, Hq, D), qs = _rows_of(q, 3, "q")
    code = _type_of(_ROPE_TYPES, q.dtype, "q")
    if out_q is None:
        out_q = _empty((T, Hq, D), q.dtype, q.device, stream)
        os_ = (Hq * D, D)
    else:
        oshape, os_ = _rows_of(out_q, 3, "out_q")
        if oshape != q.shape or out_q.dtype != q.dtype:
            raise ValueError("out_q must have q's shape and type")
    Hk, kp, ks, okp, oks = 0, None, (0, 0), None, (0, 0)
    if k is not None:
        kshape, ks = _rows_of(k, 3, "k")
        Hk = kshape[1]
        if kshape[0] != T or kshape[2] != D or k.dtype != q.dtype:
            raise ValueError("k must be [%d, Hk, %d] of q's type" % (T, D))
        if out_k is None:
            out_k = _empty(kshape, k.dtype, k.device, stream)
            oks = (Hk * D, D)
        else:
            okshape, oks = _rows_of(out_k, 3, "out_k")
            if okshape != kshape or out_k.dtype != k.dtype:
                raise ValueError("out_k must have k's shape and type")
        kp, okp = k.data_ptr(), out_k.data_ptr()
    elif out_k is not None:
        raise ValueError("out_k without k")
    half = inv_freq.numel()
    st = load().sdv_rope(T, Hq, Hk, D, 2 * half, 1 if interleaved else 0, code,
                         _stream_of(q, stream), q.data_ptr(), qs[0], qs[1], kp, ks[0], ks[1],
                         _array(positions, T, torch.int32, "positions"),
                         _array(inv_freq, half, torch.float32, "inv_freq"), factor,
                         out_q.data_ptr(), os_[0], os_[1], okp, oks[0], oks[1])
    if st != SDV_OK:
        raise SdvError(st, "sdv_rope")
    return out_q, out_k


def sdv_pages_extend(free_list: torch.Tensor, free_count: torch.Tensor, block_table: torch.Tensor,
                     held: torch.Tensor, start: torch.Tensor, N: int, page_size: int,
                     count: Optional[torch.Tensor] = None, depth: Optional[torch.Tensor] = None,
                     base: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                     slots: Optional[torch.Tensor] = None, stream=None,
                     status: Optional[torch.Tensor] = None):
    """Pages for the tokens start[b] .. start[b] + count[b] - 1 (count None: N) of
    each sequence, from the stack free_list[:free_count] into block_table [B,
    max_pages] behind the held[b] that it has; free_count and held follow (all
    int32, changed in place).  Returns (positions [B, N] int32, slots [B, N]
    int64): base[b] + start[b] + depth[b, n] (depth None: n), as sdv_rope takes
    them, and each token's place in the cache, page * page_size + place, or -1."""
    B = held.numel()
    i32 = torch.int32
    held_p = _array(held, B, i32, "held")
    if positions is None:
        positions = _empty((B, N), i32, held.device, stream)
    if slots is None:
        slots = _empty((B, N), torch.int64, held.device, stream)
    st = load().sdv_pages_extend(
        B, N, free_list.numel(), page_size, block_table.shape[1], _stream_of(held, stream),
        _array(free_list, free_list.numel(), i32, "free_list"), _array(free_count, 1, i32, "free_count"),
        _table_of(block_table, B), held_p, _array(start, B, i32, "start"),
        _array(count, B, i32, "count"), _array(depth, B * N, i32, "depth"), _array(base, B, i32, "base"),
        _array(positions, B * N, i32, "positions"), _array(slots, B * N, torch.int64, "slots"),
        _status_of(status))
    if st != SDV_OK:
        raise SdvError(st, "sdv_pages_extend")
    return positions, slots


def sdv_pages_release(free_list: torch.Tensor, free_count: torch.Tensor, block_table: torch.Tensor,
                      held: torch.Tensor, keep: torch.Tensor, page_size: int, stream=None,
                      status: Optional[torch.Tensor] = None) -> None:
    """Give back the pages behind the first keep[b] positions of each sequence
    (0: all that it holds): their entries of block_table become -1, free_list,
    free_count and held follow."""
    B = held.numel()
    i32 = torch.int32
    held_p = _array(held, B, i32, "held")
    st = load().sdv_pages_release(
        B, free_list.numel(), page_size, block_table.shape[1], _stream_of(held, stream),
        _array(free_list, free_list.numel(), i32, "free_list"), _array(free_count, 1, i32, "free_count"),
        _table_of(block_table, B), held_p, _array(keep, B, i32, "keep"),
        _status_of(status))
    if st != SDV_OK:
        raise SdvError(st, "sdv_pages_release")


def sdv_kv_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 block_table: torch.Tensor, start: torch.Tensor,
                 count: Optional[torch.Tensor] = None, k_exp: Optional[torch.Tensor] = None,
                 v_exp: Optional[torch.Tensor] = None, stream=None,
                 status: Optional[torch.Tensor] = None) -> None:
    """Write k and v [B, N, kv_heads, D] (strided views will do) at positions
    start[b] .. start[b] + count[b] - 1 of a paged cache [pages, kv_heads,
    page_size, D], quantised where its cells are float8_e4m3fn (k_exp, v_exp
    uint8 [pages, kv_heads, page_size] then hold each row's power of two)."""
    cache = _cache_of(k_cache, v_cache, k_exp, v_exp)
    (B, N, H, D), ks = _rows_of(k, 4, "k")
    vshape, vs = _rows_of(v, 4, "v")
    if vshape != k.shape or v.dtype != k.dtype or H != cache.kv_heads or D != cache.head_dim:
        raise ValueError("k and v must be [B, N, %d, %d] of one type" % (cache.kv_heads, cache.head_dim))
    code = _type_of(_HALF_TYPES, k.dtype, "k")
    st = load().sdv_kv_write(cache, B, N, code, _stream_of(k, stream), k.data_ptr(), ks[0], ks[1],
                             ks[2], v.data_ptr(), vs[0], vs[1], vs[2], _table_of(block_table, B),
                             block_table.shape[1], _array(start, B, torch.int32, "start"),
                             _array(count, B, torch.int32, "count"), _status_of(status))
    if st != SDV_OK:
        raise SdvError(st, "sdv_kv_write")


def sdv_kv_read(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                start: torch.Tensor, N: int, count: Optional[torch.Tensor] = None,
                k_exp: Optional[torch.Tensor] = None, v_exp: Optional[torch.Tensor] = None,
                dtype: Optional[torch.dtype] = None, stream=None,
                status: Optional[torch.Tensor] = None):
    """(k, v) [B, N, kv_heads, D]: positions start[b] .. start[b] + count[b] - 1
    of the cache in `dtype` (default: the cells' type, bfloat16 for e4m3); rows
    past count[b] are 0."""
    cache = _cache_of(k_cache, v_cache, k_exp, v_exp)
    if dtype is None:
        dtype = torch.bfloat16 if cache.dtype == SDV_E4M3 else k_cache.dtype
    code = _type_of(_HALF_TYPES, dtype, "dtype")
    B = start.numel()
    out = _empty((2, B, N, cache.kv_heads, cache.head_dim), dtype, k_cache.device, stream)
    st = load().sdv_kv_read(cache, B, N, code, _stream_of(k_cache, stream), out[0].data_ptr(),
                            out[1].data_ptr(), _table_of(block_table, B), block_table.shape[1],
                            _array(start, B, torch.int32, "start"),
                            _array(count, B, torch.int32, "count"), _status_of(status))
    if st != SDV_OK:
        raise SdvError(st, "sdv_kv_read")
    return out[0], out[1]


def sdv_kv_commit(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                  start: torch.Tensor, nodes: torch.Tensor, sel: torch.Tensor,
                  accept_len: torch.Tensor, k_exp: Optional[torch.Tensor] = None,
                  v_exp: Optional[torch.Tensor] = None, out_len: Optional[torch.Tensor] = None,
                  stream=None, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """After a verification step: move the accepted path's cells behind the
    prefix and return the new lengths [B] (start + 1 + accept_len).  `nodes`
    [B, K, gamma] is sdv_tree_build's; out_len=start updates it in place."""
    cache = _cache_of(k_cache, v_cache, k_exp, v_exp)
    B, K, G = nodes.shape
    if out_len is None:
        out_len = _empty((B,), torch.int32, nodes.device, stream)
    st = load().sdv_kv_commit(cache, B, K, G, _stream_of(k_cache, stream), _table_of(block_table, B),
                              block_table.shape[1], _array(start, B, torch.int32, "start"),
                              _array(nodes, B * K * G, torch.int32, "nodes"),
                              _array(sel, B, torch.int32, "sel"),
                              _array(accept_len, B, torch.int32, "accept_len"),
                              _array(out_len, B, torch.int32, "out_len"), _status_of(status))
    if st != SDV_OK:
        raise SdvError(st, "sdv_kv_commit")
    return out_len


def sdv_tree_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  block_table: torch.Tensor, ctx_len: torch.Tensor,
                  count: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                  scale: Optional[float] = None, k_exp: Optional[torch.Tensor] = None,
                  v_exp: Optional[torch.Tensor] = None, lse: bool = False,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None, status: Optional[torch.Tensor] = None):
    """Attention of the nodes q [B, N, Hq, D] of each sequence's tree over the
    cache: node i sees the ctx_len[b] committed positions and the nodes of its
    mask row ([B, N, W] or [N, W] int32 bits, sdv_tree_build's; None: a causal
    chain), whose keys and values are at positions ctx_len[b] + node.  scale
    defaults to 1 / sqrt(D).  Returns out [B, N, Hq, D], and with `lse` also the
    log-sum-exp [B, N, Hq].  `workspace` (uint8, sdv_tree_attn_workspace()
    bytes, some 40 MB) may be passed to reuse one; by default it is taken from
    torch's allocator for the call."""
    cache = _cache_of(k_cache, v_cache, k_exp, v_exp)
    (B, N, Hq, D), qs = _rows_of(q, 4, "q")
    code = _type_of(_HALF_TYPES, q.dtype, "q")
    if D != cache.head_dim:
        raise ValueError("q must be [B, N, Hq, %d]" % cache.head_dim)
    lib = load()
    handle = _stream_of(q, stream)
    mask_sb, W = 0, (N + 31) // 32
    if mask is not None:
        shape = tuple(mask.shape)
        if shape != (N, W) and shape != (B, N, W):
            raise ValueError("mask must be [%d, %d] or [%d, %d, %d]" % (N, W, B, N, W))
        mask_sb = N * W if len(shape) == 3 else 0
    out_p = _array(out, B * N * Hq * D, q.dtype, "out")
    if out is None:
        out = _empty((B, N, Hq, D), q.dtype, q.device, stream)
        out_p = out.data_ptr()
    logs = _empty((B, N, Hq), torch.float32, q.device, stream) if lse else None
    if workspace is None:
        workspace = _empty((lib.sdv_tree_attn_workspace(),), torch.uint8, q.device, stream)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous uint8")
    st = lib.sdv_tree_attn(
        cache, B, N, Hq, code, handle, q.data_ptr(), qs[0], qs[1], qs[2], _table_of(block_table, B),
        block_table.shape[1], _array(ctx_len, B, torch.int32, "ctx_len"),
        _array(count, B, torch.int32, "count"),
        None if mask is None else _array(mask, mask.numel(), torch.int32, "mask"), mask_sb,
        D ** -0.5 if scale is None else scale,
        out_p, None if logs is None else logs.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _status_of(status))
    if st != SDV_OK:
        raise SdvError(st, "sdv_tree_attn")
    return (out, logs) if lse else out


def sdv_prefix_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    prefix_table: torch.Tensor, prefix_len: torch.Tensor, block_table: torch.Tensor,
                    ctx_len: torch.Tensor, count: Optional[torch.Tensor] = None,
                    mask: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    k_exp: Optional[torch.Tensor] = None, v_exp: Optional[torch.Tensor] = None,
                    lse: bool = False, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None,
                    status: Optional[torch.Tensor] = None):
    """sdv_tree_attn for sequences that share prefixes: prefix_table [groups,
    max_prefix_pages] and prefix_len [groups] say where the prefix of each group of
    B / groups sequences lies, block_table and ctx_len what each sequence has
    added behind it, on pages of its own.  A prefix is read once for all its
    sequences.  `workspace` (uint8) has sdv_prefix_attn_workspace(B, N, Hq, D)
    bytes: some 40 MB and two or more fp32 rows for each row of out."""
    cache = _cache_of(k_cache, v_cache, k_exp, v_exp)
    (B, N, Hq, D), qs = _rows_of(q, 4, "q")
    code = _type_of(_HALF_TYPES, q.dtype, "q")
    if D != cache.head_dim:
        raise ValueError("q must be [B, N, Hq, %d]" % cache.head_dim)
    groups = prefix_len.numel()
    if groups < 1 or B % groups:
        raise ValueError("prefix_len must have a number of entries that divides %d, got %d" % (B, groups))
    lib = load()
    handle = _stream_of(q, stream)
    mask_sb, W = 0, (N + 31) // 32
    if mask is not None:
        shape = tuple(mask.shape)
        if shape != (N, W) and shape != (B, N, W):
            raise ValueError("mask must be [%d, %d] or [%d, %d, %d]" % (N, W, B, N, W))
        mask_sb = N * W if len(shape) == 3 else 0
    out_p = _array(out, B * N * Hq * D, q.dtype, "out")
    if out is None:
        out = _empty((B, N, Hq, D), q.dtype, q.device, stream)
        out_p = out.data_ptr()
    logs = _empty((B, N, Hq), torch.float32, q.device, stream) if lse else None
    if workspace is None:
        workspace = _empty((lib.sdv_prefix_attn_workspace(B, N, Hq, D),), torch.uint8, q.device, stream)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous uint8")
    st = lib.sdv_prefix_attn(
        cache, B, groups, N, Hq, code, handle, q.data_ptr(), qs[0], qs[1], qs[2],
        _table_of(prefix_table, groups), prefix_table.shape[1],
        _array(prefix_len, groups, torch.int32, "prefix_len"), _table_of(block_table, B),
        block_table.shape[1], _array(ctx_len, B, torch.int32, "ctx_len"),
        _array(count, B, torch.int32, "count"),
        None if mask is None else _array(mask, mask.numel(), torch.int32, "mask"), mask_sb,
        D ** -0.5 if scale is None else scale,
        out_p, None if logs is None else logs.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _status_of(status))
    if st != SDV_OK:
        raise SdvError(st, "sdv_prefix_attn")
    return (out, logs) if lse else out


def sdv_set_attn_test_hooks(hooks: int) -> int:
    """Fault-path test hooks of later sdv_tree_attn and sdv_prefix_attn calls
    (SDV_HOOK_ATTN_NO_COPY or 0)."""
    return load().sdv_set_attn_test_hooks(int(hooks))


def sdv_logits_process(logits: torch.Tensor, drafts: torch.Tensor,
                       counts: Optional[torch.Tensor] = None,
                       prompt: Optional[torch.Tensor] = None,
                       repetition: Optional[torch.Tensor] = None,
                       frequency: Optional[torch.Tensor] = None,
                       presence: Optional[torch.Tensor] = None,
                       bias_ids: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, allow: Optional[torch.Tensor] = None,
                       rows: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       stream=None, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The sampling parameters of every draft position, on verifier logits
    [B, K, gamma + 1, V], or with rows [B, K, gamma + 1] (sdv_tree_build's) on a
    tree's logits [B, nodes, V]: penalties that count the history (counts [B, V]
    int32, prompt bits [B, ceil(V / 32)] int32) and the draft's earlier tokens,
    biases [B, M], and a grammar's allowed tokens (bits [B, K, gamma + 1,
    ceil(V / 32)] int32).  Returns [B, K, gamma + 1, V] for a Verifier call;
    out=logits works in place when rows is None."""
    B, K, G = drafts.shape
    V = logits.shape[-1]
    code = _dtype_code(logits.dtype)
    W = (V + 31) // 32
    nsrc = 0
    if rows is None:
        if tuple(logits.shape) != (B, K, G + 1, V):
            raise ValueError("logits must be [%d, %d, %d, V]" % (B, K, G + 1))
    else:
        if logits.dim() != 3 or logits.shape[0] != B:
            raise ValueError("logits must be [%d, nodes, V]" % B)
        nsrc = logits.shape[1]
    M = 0
    if bias_ids is not None or bias is not None:
        if bias_ids is None or bias is None or bias_ids.numel() != bias.numel() or bias_ids.numel() % B:
            raise ValueError("bias_ids and bias must be [%d, M] both" % B)
        M = bias_ids.numel() // B
    if out is None:
        out = _empty((B, K, G + 1, V), logits.dtype, logits.device, stream)
    i32, f32 = torch.int32, torch.float32
    st = load().sdv_logits_process(
        B, K, G, V, code, _stream_of(logits, stream), _array(logits, logits.numel(), logits.dtype, "logits"),
        nsrc, _array(rows, B * K * (G + 1), i32, "rows"), _array(drafts, B * K * G, i32, "drafts"),
        _array(counts, B * V, i32, "counts"), _array(prompt, B * W, i32, "prompt"),
        _array(repetition, B, f32, "repetition"), _array(frequency, B, f32, "frequency"),
        _array(presence, B, f32, "presence"), M, _array(bias_ids, B * M, i32, "bias_ids") if M else None,
        _array(bias, B * M, f32, "bias") if M else None,
        _array(allow, B * K * (G + 1) * W, i32, "allow"),
        _array(out, B * K * (G + 1) * V, logits.dtype, "out"), _status_of(status))
    if st != SDV_OK:
        raise SdvError(st, "sdv_logits_process")
    return out


def sdv_counts_commit(counts: torch.Tensor, drafts: torch.Tensor, sel: torch.Tensor,
                      accept_len: torch.Tensor, next_token: torch.Tensor, stream=None,
                      status: Optional[torch.Tensor] = None) -> None:
    """Add a verification step's committed tokens (the accepted ones and the
    next token) to counts [B, V] int32."""
    B, K, G = drafts.shape
    V = counts.shape[-1]
    i32 = torch.int32
    st = load().sdv_counts_commit(B, K, G, V, _stream_of(counts, stream),
                                  _array(drafts, B * K * G, i32, "drafts"), _array(sel, B, i32, "sel"),
                                  _array(accept_len, B, i32, "accept_len"),
                                  _array(next_token, B, i32, "next_token"),
                                  _array(counts, B * V, i32, "counts"), _status_of(status))
    if st != SDV_OK:
        raise SdvError(st, "sdv_counts_commit")


def _logit_rows(t: torch.Tensor, name: str):
    """(B, rows per entry of the first dimension, V, elements between rows) of
    logits [B, ..., V] whose rows are evenly apart."""
    shape, stride = t.shape, t.stride()
    if len(shape) < 2:
        raise ValueError("%s must be [B, ..., V], got %s" % (name, tuple(shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if stride[-1] != 1 and shape[-1] != 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)
    if 0 in shape:
        return shape[0], 1, shape[-1], shape[-1]
    rows, step = 1, None                 # of the dimensions from here on
    for n, s in zip(shape[-2::-1], stride[-2::-1]):
        if n == 1:
            continue
        if step is None:
            step = s
        elif s != rows * step:
            raise ValueError("the rows of %s must be evenly apart" % name)
        rows *= n
    return shape[0], rows // shape[0], shape[-1], shape[-1] if step is None else step


def _cuts(B: int, temperature, top_k, top_p, min_p):
    f32 = torch.float32
    return (_array(temperature, B, f32, "temperature"), _array(top_k, B, torch.int32, "top_k"),
            _array(top_p, B, f32, "top_p"), _array(min_p, B, f32, "min_p"))


def sdv_sample(logits: torch.Tensor, uniform: torch.Tensor, temperature: Optional[torch.Tensor] = None,
               top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
               min_p: Optional[torch.Tensor] = None, logprob: bool = False,
               tokens: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None, stream=None,
               status: Optional[torch.Tensor] = None):
    """A token for each row of logits [B, ..., V] (bfloat16 or float32) from the
    random numbers uniform [B, ...] in [0, 1), under the parameters of its sequence
    ([B] each; temperature 0 takes the best token): tokens [B, ...] int32, and with
    `logprob` also their log-probabilities among what is kept.  `kept` (int32
    [B, ...]) receives how many tokens that is."""
    B, per, V, step = _logit_rows(logits, "logits")
    code = _dtype_code(logits.dtype)
    shape = logits.shape[:-1]
    rows = B * per if logits.numel() else 0
    if tokens is None:
        tokens = _empty(shape, torch.int32, logits.device, stream)
    logs = _empty(shape, torch.float32, logits.device, stream) if logprob else None
    st = load().sdv_sample(rows, per, V, code, _stream_of(logits, stream), logits.data_ptr(), step,
                           *_cuts(B, temperature, top_k, top_p, min_p),
                           _array(uniform, rows, torch.float32, "uniform"),
                           _array(tokens, rows, torch.int32, "tokens"),
                           None if logs is None else logs.data_ptr(),
                           _array(kept, rows, torch.int32, "kept"), _status_of(status))
    if st != SDV_OK:
        raise SdvError(st, "sdv_sample")
    return (tokens, logs) if logprob else tokens


def sdv_logits_truncate(logits: torch.Tensor, temperature: Optional[torch.Tensor] = None,
                        top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
                        min_p: Optional[torch.Tensor] = None, kept: bool = False,
                        out: Optional[torch.Tensor] = None, stream=None,
                        status: Optional[torch.Tensor] = None):
    """logits [B, ..., V] with -inf in the place of every token that sdv_sample
    under the same parameters would not draw (not scaled by the temperature), for a
    Verifier call that is lossless for the truncated distribution; with `kept` also
    how many are left [B, ...].  out=logits works in place."""
    B, per, V, step = _logit_rows(logits, "logits")
    code = _dtype_code(logits.dtype)
    rows = B * per if logits.numel() else 0
    if out is None:
        out = _empty(logits.shape, logits.dtype, logits.device, stream)
        out_step = V
    else:
        if out.shape != logits.shape or out.dtype != logits.dtype:
            raise ValueError("out must have the shape and type of logits")
        out_step = _logit_rows(out, "out")[3]
    many = _empty(logits.shape[:-1], torch.int32, logits.device, stream) if kept else None
    st = load().sdv_logits_truncate(rows, per, V, code, _stream_of(logits, stream), logits.data_ptr(), step,
                                    *_cuts(B, temperature, top_k, top_p, min_p), out.data_ptr(), out_step,
                                    None if many is None else many.data_ptr(), _status_of(status))
    if st != SDV_OK:
        raise SdvError(st, "sdv_logits_truncate")
    return (out, many) if kept else out
