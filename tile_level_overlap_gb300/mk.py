"""Thin Python binding of libmk's C ABI (include/mk.h).

Argument marshalling only: every step of the forward pass runs in the CUDA
kernels of libmk.  Tensors are passed as raw device pointers; PyTorch is used
for device memory and streams.  There is no fallback: if libmk.so is missing
or no GPU is present, the calls raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmk.so")

MK_OK = 0
MK_ERR_INVALID_ARG = 1
MK_ERR_CUDA = 2
MK_ERR_TIMEOUT = 3
MK_ERR_BOUNDS = 4
MK_ERR_UNSUPPORTED = 5
MK_ERR_NO_DEVICE = 6
MK_DECODE = 0
MK_PREFILL = 1
MK_LM_FUSED, MK_LM_SEPARATE = 0, 1
MK_BF16, MK_FP16 = 0, 1
MK_PAGED_MAX_REQUESTS = 4096
MK_PAGED_WORKSPACE_BYTES = 64 << 20  # scratch of mk_paged_attention
TRACE_WORDS = 16  # u64 words per trace record (mk_trace_copy)
MK_NOALLOC_SCRATCH_BYTES = 16 << 20  # static device scratch of mk_decode_step_noalloc

EXPORTED = [
    "mk_plan_create", "mk_plan_destroy", "mk_kv_cache_bytes", "mk_decode_step",
    "mk_decode_step_host", "mk_prefill", "mk_run_per_op", "mk_status", "mk_plan_reset",
    "mk_status_string", "mk_plan_get_stats", "mk_plan_check", "mk_plan_set_debug",
    "mk_trace_copy", "mk_plan_debug_drop_release", "mk_debug_gemm_bf16", "mk_decode_step_noalloc",
    "mk_plan_set_lm_mode", "mk_decode_steps", "mk_prefill_logits", "mk_prefill_batch",
    "mk_decode_step_slots", "mk_plan_create_for_sms", "mk_prefill_chunks",
    "mk_paged_tables", "mk_rope_init", "mk_paged_append", "mk_paged_attention",
]


class mk_model_cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("n_layers", "hidden", "n_q_heads", "n_kv_heads", "head_dim", "ffn", "vocab")] + [
        ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float),
        ("qk_norm", ctypes.c_int), ("tied_embeddings", ctypes.c_int)]


_PP = ctypes.POINTER(ctypes.c_void_p)


class mk_weight_ptrs(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p),
                ("lm_head", ctypes.c_void_p)] + [(n, _PP) for n in (
                    "attn_norm", "wq", "wk", "wv", "wo", "q_norm", "k_norm", "ffn_norm",
                    "w_gate", "w_up", "w_down")]


class mk_plan_stats(ctypes.Structure):
    _fields_ = [("n_instr_decode", ctypes.c_uint32), ("n_instr_prefill", ctypes.c_uint32),
                ("n_barriers", ctypes.c_uint32), ("n_launches_per_op_decode", ctypes.c_uint32),
                ("n_ctas", ctypes.c_uint32), ("n_splits", ctypes.c_uint32),
                ("weight_bytes", ctypes.c_uint64), ("scratch_bytes", ctypes.c_uint64),
                ("decode_path", ctypes.c_uint32), ("queue_hash", ctypes.c_uint64)]


class mk_paged_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "workspace", "status")] + [
        (n, ctypes.c_int64) for n in ("page_stride", "head_stride", "token_stride")] + [
        (n, ctypes.c_int) for n in ("n_q_heads", "n_kv_heads", "head_dim", "page_size", "n_pages",
                                    "dtype")]


class mk_paged_batch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("block_table", "cu_new", "kv_lens", "positions",
                                               "slots")] + [
        (n, ctypes.c_int) for n in ("n", "max_blocks", "max_tokens", "max_new", "page_size")]


class mk_rope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("n_axes", ctypes.c_int),
                ("turn", ctypes.c_uint64 * 64), ("axis", ctypes.c_uint8 * 64)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmk.so (built by tile_level_overlap_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with tile_level_overlap_gb300.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32p, f32p = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
    L.mk_plan_create.argtypes = [ctypes.POINTER(mk_model_cfg), ctypes.POINTER(mk_weight_ptrs),
                                 ctypes.c_int, ctypes.c_int, ctypes.POINTER(vp)]
    L.mk_plan_create_for_sms.argtypes = [ctypes.POINTER(mk_model_cfg), ctypes.POINTER(mk_weight_ptrs),
                                         ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(vp)]
    L.mk_plan_destroy.argtypes = [vp]
    L.mk_plan_destroy.restype = None
    L.mk_kv_cache_bytes.argtypes = [vp]
    L.mk_kv_cache_bytes.restype = ctypes.c_size_t
    L.mk_decode_step.argtypes = [vp, i32p, i32p, ctypes.c_int, vp, f32p, vp]
    L.mk_decode_step_host.argtypes = [vp, i32p, i32p, ctypes.c_int, vp, f32p, vp]
    L.mk_prefill.argtypes = [vp, i32p, ctypes.c_int, vp, f32p, vp]
    L.mk_run_per_op.argtypes = [vp, ctypes.c_int, ctypes.c_int, i32p, i32p, ctypes.c_int, vp, f32p, vp]
    L.mk_status.argtypes = [vp, vp]
    L.mk_plan_reset.argtypes = [vp, vp]
    L.mk_status_string.argtypes = [ctypes.c_int]
    L.mk_status_string.restype = ctypes.c_char_p
    L.mk_plan_get_stats.argtypes = [vp, ctypes.POINTER(mk_plan_stats)]
    L.mk_plan_check.argtypes = [ctypes.POINTER(mk_model_cfg), ctypes.c_int, ctypes.c_int,
                                ctypes.c_uint64, ctypes.POINTER(mk_plan_stats)]
    L.mk_plan_set_debug.argtypes = [vp, ctypes.c_int, ctypes.c_uint64, ctypes.c_int, ctypes.c_uint64]
    L.mk_plan_set_lm_mode.argtypes = [vp, ctypes.c_int]
    L.mk_decode_steps.argtypes = [vp, vp, vp, ctypes.c_int, vp, vp, vp, vp]
    L.mk_prefill_logits.argtypes = [vp, vp, ctypes.c_int, vp, vp, vp]
    L.mk_decode_step_slots.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, vp, vp]
    L.mk_prefill_batch.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int32), ctypes.c_int, ctypes.c_int,
                                   vp, vp, vp]
    L.mk_prefill_chunks.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int32), ctypes.c_int, vp, vp, vp]
    L.mk_trace_copy.argtypes = [vp, vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)]
    L.mk_plan_debug_drop_release.argtypes = [vp, ctypes.c_uint32]
    L.mk_debug_gemm_bf16.argtypes = [vp, vp, vp, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                     ctypes.c_int, vp]
    L.mk_decode_step_noalloc.argtypes = [ctypes.POINTER(mk_model_cfg), ctypes.POINTER(mk_weight_ptrs),
                                         ctypes.c_int, ctypes.c_int, i32p, i32p, ctypes.c_int, vp,
                                         f32p, vp]
    i64 = ctypes.c_int64
    L.mk_paged_tables.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, vp, vp, vp]
    L.mk_rope_init.argtypes = [vp, ctypes.c_int, ctypes.c_double, vp, ctypes.c_int, vp]
    L.mk_paged_append.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, ctypes.c_float, vp,
                                  vp, i64, vp, ctypes.c_int, vp]
    L.mk_paged_attention.argtypes = [vp, vp, vp, i64, vp, i64, vp, ctypes.c_float, ctypes.c_int, vp]
    _lib = L
    return L


class MkError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {lib().mk_status_string(code).decode()} (code {code})")


def _check(code: int, what: str) -> None:
    if code != MK_OK:
        raise MkError(code, what)


def model_cfg(cfg) -> mk_model_cfg:
    return mk_model_cfg(cfg.n_layers, cfg.hidden, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim,
                        cfg.ffn, cfg.vocab, float(cfg.rms_eps), float(cfg.rope_theta),
                        int(bool(cfg.qk_norm)), int(bool(cfg.tied_embeddings)))


def plan_check(cfg, max_batch: int, max_ctx: int, seed: int = 0):
    """Host-only plan build + simulation; returns (status, stats)."""
    st = mk_plan_stats()
    rc = lib().mk_plan_check(ctypes.byref(model_cfg(cfg)), max_batch, max_ctx, seed, ctypes.byref(st))
    return rc, st


def weight_ptrs(cfg, weights):
    """mk_weight_ptrs over name -> torch bf16 CUDA tensor; returns (struct,
    keep-alive list of the pointer arrays it references)."""
    n = cfg.n_layers
    keep = []
    wp = mk_weight_ptrs()
    wp.embed = _ptr(weights["embed"])
    wp.final_norm = _ptr(weights["final_norm"])
    wp.lm_head = _ptr(weights["lm_head"]) if "lm_head" in weights else None
    for k in ("attn_norm", "wq", "wk", "wv", "wo", "q_norm", "k_norm", "ffn_norm", "w_gate", "w_up",
              "w_down"):
        if all(f"layers.{l}.{k}" in weights for l in range(n)):
            a = (ctypes.c_void_p * n)(*[_ptr(weights[f"layers.{l}.{k}"]) for l in range(n)])
            keep.append(a)
            setattr(wp, k, ctypes.cast(a, _PP))
    return wp, keep


def decode_step_noalloc(cfg, weights, max_batch: int, max_ctx: int, tokens, positions, kv, logits,
                        stream=None) -> int:
    """mk_decode_step_noalloc: one decode step using only the library's static
    device scratch (no device allocation).  Returns the C status code."""
    wp, keep = weight_ptrs(cfg, weights)
    rc = lib().mk_decode_step_noalloc(ctypes.byref(model_cfg(cfg)), ctypes.byref(wp), max_batch,
                                      max_ctx, _ptr(tokens), _ptr(positions), int(tokens.numel()),
                                      _ptr(kv), _ptr(logits), _stream_ptr(stream))
    del keep
    return rc


def _stream_ptr(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _ptr(t) -> int:
    return int(t.data_ptr())


class Plan:
    """A plan over weights held as torch bf16 CUDA tensors (name -> tensor, as
    produced by synth.make_weights).  Keeps references so the weights outlive
    the plan."""

    def __init__(self, cfg, weights: Dict[str, "object"], max_batch: int, max_ctx: int,
                 n_sms: int = 0):
        """n_sms > 0 (test-only): tile and launch the plan as on a device with
        that many SMs (mk_plan_create_for_sms)."""
        L = lib()
        self.cfg = cfg
        self.max_batch = max_batch
        self.max_ctx = max_ctx
        self._w = weights
        n = cfg.n_layers

        def arr(key):
            if not all(f"layers.{l}.{key}" in weights for l in range(n)):
                return None
            a = (ctypes.c_void_p * n)(*[_ptr(weights[f"layers.{l}.{key}"]) for l in range(n)])
            return a

        self._arrays = {k: arr(k) for k in ("attn_norm", "wq", "wk", "wv", "wo", "q_norm", "k_norm",
                                            "ffn_norm", "w_gate", "w_up", "w_down")}
        wp = mk_weight_ptrs()
        wp.embed = _ptr(weights["embed"])
        wp.final_norm = _ptr(weights["final_norm"])
        wp.lm_head = _ptr(weights["lm_head"]) if "lm_head" in weights else None
        for k, a in self._arrays.items():
            setattr(wp, k, ctypes.cast(a, _PP) if a is not None else None)
        h = ctypes.c_void_p()
        _check(L.mk_plan_create_for_sms(ctypes.byref(model_cfg(cfg)), ctypes.byref(wp), max_batch,
                                        max_ctx, int(n_sms), ctypes.byref(h)), "mk_plan_create")
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            lib().mk_plan_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---- sizes
    def kv_cache_bytes(self) -> int:
        return int(lib().mk_kv_cache_bytes(self.h))

    def stats(self) -> mk_plan_stats:
        st = mk_plan_stats()
        _check(lib().mk_plan_get_stats(self.h, ctypes.byref(st)), "mk_plan_get_stats")
        return st

    # ---- steps (device tensors)
    def decode_step(self, tokens, positions, kv, logits, stream=None) -> None:
        _check(lib().mk_decode_step(self.h, _ptr(tokens), _ptr(positions), int(tokens.numel()),
                                    _ptr(kv), _ptr(logits), _stream_ptr(stream)), "mk_decode_step")

    def decode_steps(self, token, position, n_steps: int, kv, out_tokens, logits, stream=None) -> None:
        """mk_decode_steps: n_steps greedy decode steps of one sequence in one
        launch (device tensors: token [1], position [1], out_tokens [n_steps],
        logits [V])."""
        _check(lib().mk_decode_steps(self.h, _ptr(token), _ptr(position), int(n_steps), _ptr(kv),
                                     _ptr(out_tokens), _ptr(logits), _stream_ptr(stream)),
               "mk_decode_steps")

    def decode_step_slots(self, tokens, positions, slots, kv, logits, stream=None) -> None:
        """mk_decode_step_slots: column c is tokens[c] of cache slot slots[c] at
        positions[c] (a prompt chunk = several columns of one slot)."""
        _check(lib().mk_decode_step_slots(self.h, _ptr(tokens), _ptr(positions), _ptr(slots),
                                          int(tokens.numel()), _ptr(kv), _ptr(logits),
                                          _stream_ptr(stream)), "mk_decode_step_slots")

    def decode_step_host(self, tokens, positions, kv, logits, stream=None) -> int:
        """tokens/positions/logits are CPU tensors (pinned for speed)."""
        return lib().mk_decode_step_host(self.h, _ptr(tokens), _ptr(positions), int(tokens.numel()),
                                         _ptr(kv), _ptr(logits), _stream_ptr(stream))

    def prefill(self, tokens, kv, logits, stream=None) -> None:
        _check(lib().mk_prefill(self.h, _ptr(tokens), int(tokens.numel()), _ptr(kv), _ptr(logits),
                                _stream_ptr(stream)), "mk_prefill")

    def prefill_batch(self, tokens, lens, kv, logits, stream=None) -> None:
        """mk_prefill_batch: tokens device [batch, stride], lens a list of
        prompt lengths, logits device [batch, V]; prompt b to cache slot b."""
        n = len(lens)
        arr = (ctypes.c_int32 * n)(*[int(v) for v in lens])
        _check(lib().mk_prefill_batch(self.h, _ptr(tokens), arr, n, int(tokens.shape[1]), _ptr(kv),
                                      _ptr(logits), _stream_ptr(stream)), "mk_prefill_batch")

    def prefill_chunks(self, tokens, chunks, kv, logits, stream=None) -> None:
        """mk_prefill_chunks: tokens device int32 [*], chunks a list of (slot,
        pos0, len, token offset), logits device [n, V]."""
        n = len(chunks)
        flat = [int(v) for c in chunks for v in c]
        arr = (ctypes.c_int32 * (4 * n))(*flat)
        _check(lib().mk_prefill_chunks(self.h, _ptr(tokens), arr, n, _ptr(kv), _ptr(logits),
                                       _stream_ptr(stream)), "mk_prefill_chunks")

    def prefill_logits(self, tokens, kv, logits, stream=None) -> None:
        """mk_prefill_logits: the prompt's logits for every token, [len, V]."""
        _check(lib().mk_prefill_logits(self.h, _ptr(tokens), int(tokens.numel()), _ptr(kv),
                                       _ptr(logits), _stream_ptr(stream)), "mk_prefill_logits")

    def run_per_op(self, mode: int, tokens, positions, kv, logits, use_graph: bool = False,
                   stream=None) -> None:
        n = int(tokens.numel())
        _check(lib().mk_run_per_op(self.h, mode, int(use_graph), _ptr(tokens),
                                   _ptr(positions) if positions is not None else None, n,
                                   _ptr(kv), _ptr(logits), _stream_ptr(stream)), "mk_run_per_op")

    def status(self, stream=None) -> int:
        return lib().mk_status(self.h, _stream_ptr(stream))

    def reset(self, stream=None) -> None:
        _check(lib().mk_plan_reset(self.h, _stream_ptr(stream)), "mk_plan_reset")

    def set_debug(self, force_ctas: int = 0, queue_perm_seed: int = 0, trace: bool = False,
                  wait_limit_ns: int = 0) -> None:
        _check(lib().mk_plan_set_debug(self.h, force_ctas, queue_perm_seed, int(trace), wait_limit_ns),
               "mk_plan_set_debug")

    def set_lm_mode(self, mode: int) -> None:
        """MK_LM_FUSED: the LM head inside the persistent step; MK_LM_SEPARATE:
        the layers persistent, then the LM head as a kernel-per-operator launch."""
        _check(lib().mk_plan_set_lm_mode(self.h, mode), "mk_plan_set_lm_mode")

    def debug_drop_release(self, index: int) -> None:
        _check(lib().mk_plan_debug_drop_release(self.h, index), "mk_plan_debug_drop_release")

    def trace(self):
        """Trace records of the last traced launch as a numpy structured array."""
        import numpy as np
        n = self.stats().n_instr_decode
        buf = np.zeros(n * TRACE_WORDS, dtype=np.uint64)
        got = ctypes.c_size_t()
        _check(lib().mk_trace_copy(self.h, buf.ctypes.data, buf.nbytes, ctypes.byref(got)), "mk_trace_copy")
        rec = buf[: got.value * TRACE_WORDS].reshape(-1, TRACE_WORDS)
        return rec


# ---------------------------------------------------------------- paged KV cache

def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _on_gpu(t, dtype, what: str) -> None:
    _need(t.is_cuda and t.dtype == dtype, f"{what}: a CUDA tensor of {dtype} is wanted")


def _int32(t, what: str) -> None:
    import torch
    _on_gpu(t, torch.int32, what)
    _need(t.is_contiguous(), f"{what}: contiguous")


def _heads(t, n_heads: int, dim: int, dtype, device, what: str) -> int:
    """Stride from token to token of a [tokens, heads, head_dim] tensor whose
    heads lie end to end."""
    _on_gpu(t, dtype, what)
    s = t.stride()
    _need(t.device == device and t.dim() == 3 and t.shape[1] == n_heads and t.shape[2] == dim
          and s[2] == 1 and (n_heads == 1 or s[1] == dim),
          f"{what}: [tokens, {n_heads}, {dim}] with contiguous heads on the cache's device")
    return s[0] if t.shape[0] > 1 else max(s[0], n_heads * dim)


def _run_on(device, stream):
    """(device guard or None, raw stream) of a call on `device`'s tensors: the
    given stream or the device's current one."""
    import torch
    raw = (int(stream.cuda_stream) if stream is not None
           else torch.cuda.current_stream(device).cuda_stream)
    return (None if torch.cuda.current_device() == device.index else torch.cuda.device(device)), raw


def _call(device, stream, what: str, fn, *args) -> None:
    guard, raw = _run_on(device, stream)
    if guard is None:
        rc = fn(*args, raw)
    else:
        with guard:
            rc = fn(*args, raw)
    if rc != MK_OK:
        raise MkError(rc, what)


class Rope:
    """Rotary positions (mk_rope).  One axis, or several: `sections` gives the
    pairs each axis turns, one section after another, or with interleaved=True
    the axes in turn (pair i on axis i % n_axes while that axis has pairs left,
    else on axis 0); `axis_of_pair` names each pair's axis outright.  inv_freq
    (radians per position, one per pair) replaces theta^(-2i / rotary_dim)."""

    def __init__(self, head_dim: int, theta: float = 10000.0, rotary_dim: Optional[int] = None,
                 sections=None, interleaved: bool = False, axis_of_pair=None, inv_freq=None):
        rot = head_dim if rotary_dim is None else int(rotary_dim)
        half = rot // 2
        if axis_of_pair is None and sections is not None:
            _need(sum(sections) == half, "sections: rotary_dim / 2 pairs in all are wanted")
            n = len(sections)
            if interleaved:
                axis_of_pair = [i % n if i // n < sections[i % n] else 0 for i in range(half)]
            else:
                axis_of_pair = [a for a, k in enumerate(sections) for _ in range(k)]
            self.n_axes = n
        else:
            self.n_axes = 1 if axis_of_pair is None else max(axis_of_pair) + 1
        _need(axis_of_pair is None or len(axis_of_pair) == half, "axis_of_pair: one per pair")
        _need(inv_freq is None or len(inv_freq) == half, "inv_freq: one per pair")
        _need(rot <= head_dim, "rotary_dim: at most head_dim")
        self.c = mk_rope()
        axes = None if axis_of_pair is None else (ctypes.c_uint8 * half)(*[int(a) for a in axis_of_pair])
        freq = None if inv_freq is None else (ctypes.c_double * half)(*[float(f) for f in inv_freq])
        _check(lib().mk_rope_init(ctypes.byref(self.c), rot, float(theta), freq, self.n_axes, axes),
               "mk_rope_init")
        self._p = ctypes.addressof(self.c)


class PagedBatch:
    """The tables of a step (mk_paged_batch) over torch int32 CUDA tensors:
    block_table [n, max_blocks], cu_new [n + 1], kv_lens [n], and for build()
    and append positions and slots [max_tokens].  Holds references to them."""

    def __init__(self, block_table, cu_new, kv_lens, positions=None, slots=None, *, page_size: int,
                 max_new: int):
        for name, t in (("block_table", block_table), ("cu_new", cu_new), ("kv_lens", kv_lens),
                        ("positions", positions), ("slots", slots)):
            if t is not None:
                _int32(t, name)
                _need(t.device == kv_lens.device, f"{name}: on one device with kv_lens")
        n = kv_lens.numel()
        _need(block_table.dim() == 2 and block_table.shape[0] == n and cu_new.numel() == n + 1,
              "block_table [n, max_blocks], cu_new [n + 1], kv_lens [n]")
        _need((positions is None) == (slots is None) and
              (slots is None or positions.numel() == slots.numel()), "positions and slots of one length")
        self.block_table, self.cu_new, self.kv_lens = block_table, cu_new, kv_lens
        self.positions, self.slots = positions, slots
        self.n, self.device, self.page_size, self.max_new = n, kv_lens.device, page_size, int(max_new)
        self.max_tokens = 0 if slots is None else slots.numel()
        self.c = mk_paged_batch(_ptr(block_table), _ptr(cu_new), _ptr(kv_lens),
                                None if slots is None else _ptr(positions),
                                None if slots is None else _ptr(slots), n, block_table.shape[1],
                                self.max_tokens, self.max_new, page_size)
        self._p = ctypes.addressof(self.c)

    def build(self, ctx_lens, new_lens, free_pages, n_free, n_left, status=None, stream=None) -> None:
        """mk_paged_tables: fill the tables from device int32 lengths [n], taking
        pages from the end of free_pages[0 : n_free[0]]; n_left[0] receives what
        remains."""
        _need(self.slots is not None, "build needs positions and slots")
        for name, t, k in (("ctx_lens", ctx_lens, self.n), ("new_lens", new_lens, self.n),
                           ("free_pages", free_pages, None), ("n_free", n_free, 1),
                           ("n_left", n_left, 1), ("status", status, 1)):
            if t is not None:
                _int32(t, name)
                _need(t.device == self.device and (k is None or t.numel() == k),
                      f"{name}: {k} values on the batch's device")
        self.c.max_tokens = self.max_tokens
        _call(self.device, stream, "mk_paged_tables", lib().mk_paged_tables, self._p, _ptr(ctx_lens),
              _ptr(new_lens), _ptr(free_pages), free_pages.numel(), _ptr(n_free), _ptr(n_left),
              None if status is None else _ptr(status))


class PagedCache:
    """One layer's paged cache (mk_paged_cache) over torch tensors k and v
    [n_pages, n_kv_heads, page_size, head_dim] of bf16 or fp16 (any view of that
    shape with contiguous head_dim, equal strides for both).  `workspace`
    (uint8, MK_PAGED_WORKSPACE_BYTES) may be shared by caches whose calls do not
    overlap; without one the first attention call allocates it.  Holds
    references to the tensors."""

    def __init__(self, k, v, n_q_heads: int, workspace=None):
        import torch
        _need(k.is_cuda and v.is_cuda and k.device == v.device and k.dtype == v.dtype
              and k.dtype in (torch.bfloat16, torch.float16), "k, v: CUDA tensors of bf16 or fp16")
        _need(k.dim() == 4 and k.shape == v.shape and k.stride() == v.stride() and k.stride(3) == 1,
              "k, v: [n_pages, n_kv_heads, page_size, head_dim], same strides")
        n_pages, hkv, page, d = k.shape
        self.k, self.v, self.device, self.dtype = k, v, k.device, k.dtype
        self.n_q_heads, self.n_kv_heads, self.head_dim, self.page_size = n_q_heads, hkv, d, page
        self._status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self.workspace = None
        s = k.stride()
        self.c = mk_paged_cache(_ptr(k), _ptr(v), None, _ptr(self._status), s[0], s[1], s[2],
                                n_q_heads, hkv, d, page, n_pages,
                                MK_BF16 if k.dtype == torch.bfloat16 else MK_FP16)
        self._p = ctypes.addressof(self.c)
        if workspace is not None:
            _need(workspace.device == k.device and workspace.is_contiguous() and
                  workspace.numel() * workspace.element_size() >= MK_PAGED_WORKSPACE_BYTES,
                  "workspace: MK_PAGED_WORKSPACE_BYTES on the cache's device")
            self._set_workspace(workspace)

    def _set_workspace(self, t) -> None:
        self.workspace = t
        self.c.workspace = _ptr(t)

    def append(self, q, k, v, slots, positions=None, rope: Optional[Rope] = None, q_out=None,
               q_norm=None, k_norm=None, eps: float = 1e-6, stream=None) -> None:
        """mk_paged_append: q [T, n_q_heads, head_dim], k, v [T, n_kv_heads,
        head_dim], slots int32 [T], positions int32 [T] or [n_axes, T]; q_out
        defaults to q itself."""
        q_out = q if q_out is None else q_out
        hq, hkv, d, dev, typ = self.n_q_heads, self.n_kv_heads, self.head_dim, self.device, self.dtype
        n = q.shape[0]
        _int32(slots, "slots")
        _need(slots.numel() == n and k.shape[0] == n and v.shape[0] == n and q_out.shape[0] == n
              and slots.device == dev, "q, k, v, q_out and slots of one length and device")
        for name, g in (("q_norm", q_norm), ("k_norm", k_norm)):
            if g is not None:
                _on_gpu(g, typ, name)
                _need(g.numel() == d and g.is_contiguous() and g.device == dev, f"{name}: [{d}]")
        pos = pos_stride = 0
        if rope is not None:
            _need(positions is not None, "rope needs positions")
            _on_gpu(positions, self._status.dtype, "positions")
            one = positions.dim() == 1
            _need(positions.shape[-1] == n and positions.device == dev and positions.dim() <= 2 and
                  (1 if one else positions.shape[0]) == rope.n_axes and (n < 2 or positions.stride(-1) == 1),
                  f"positions: [{rope.n_axes}, {n}]")
            pos, pos_stride = _ptr(positions), 0 if one else positions.stride(0)
        qs, ks, vs, os = (_heads(q, hq, d, typ, dev, "q"), _heads(k, hkv, d, typ, dev, "k"),
                          _heads(v, hkv, d, typ, dev, "v"), _heads(q_out, hq, d, typ, dev, "q_out"))
        if n == 0:
            return
        _call(dev, stream, "mk_paged_append", lib().mk_paged_append, self._p, _ptr(q), qs, _ptr(k), ks,
              _ptr(v), vs, _ptr(q_out), os, None if q_norm is None else _ptr(q_norm),
              None if k_norm is None else _ptr(k_norm), eps, None if rope is None else rope._p,
              pos or None, pos_stride, _ptr(slots), n)

    def attention(self, q, batch: PagedBatch, out, lse=None, scale: float = 0.0, window: int = 0,
                  stream=None) -> None:
        """mk_paged_attention: q, out [rows, n_q_heads, head_dim], lse float32
        [rows, n_q_heads] or None."""
        import torch
        if self.workspace is None:
            self._set_workspace(torch.empty(MK_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device=self.device))
        hq, d, dev, typ = self.n_q_heads, self.head_dim, self.device, self.dtype
        n = q.shape[0]
        _need(out.shape[0] == n and batch.device == dev, "q, out and batch of one length and device")
        if lse is not None:
            _on_gpu(lse, torch.float32, "lse")
            _need(lse.is_contiguous() and lse.numel() == n * hq and lse.device == dev, f"lse: [{n}, {hq}]")
        qs, os = _heads(q, hq, d, typ, dev, "q"), _heads(out, hq, d, typ, dev, "out")
        if n == 0:
            return
        batch.c.max_tokens = n
        _call(dev, stream, "mk_paged_attention", lib().mk_paged_attention, self._p, batch._p, _ptr(q), qs,
              _ptr(out), os, None if lse is None else _ptr(lse), scale, window)

    def status(self) -> int:
        """The status word (waits for the device work that writes it)."""
        return int(self._status.item())

    def reset(self) -> None:
        self._status.zero_()
