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
MK_PAGED_MAX_HEADS = 65536
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
# A step makes these calls per layer, and the smallest take the GPU a few
# microseconds: the checks of a call are one expression each, and what is wrong
# is worked out after one has failed.

def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _tensors(device, **wanted):
    """Raise for the first of name=(tensor, dtype, shape or None) that is not a
    contiguous tensor of that kind on `device`."""
    for name, (t, dtype, shape) in wanted.items():
        if t is None:
            continue
        _need(t.is_cuda and t.device == device, f"{name}: a CUDA tensor on {device} is wanted")
        _need(t.dtype == dtype, f"{name}: {dtype} is wanted, not {t.dtype}")
        _need(shape is None or tuple(t.shape) == shape, f"{name}: {shape} is wanted, not {tuple(t.shape)}")
        _need(t.is_contiguous(), f"{name}: contiguous")


def _heads(device, dtype, **wanted):
    """Raise for the first of name=(tensor, shape) that is not [tokens, heads,
    head_dim] with heads that lie end to end."""
    for name, (t, shape) in wanted.items():
        _need(t.is_cuda and t.device == device and t.dtype == dtype and tuple(t.shape) == shape,
              f"{name}: {dtype} {shape} on {device} is wanted, not {t.dtype} {tuple(t.shape)} on {t.device}")
        s = t.stride()
        _need(s[2] == 1 and (shape[1] == 1 or s[1] == shape[2]), f"{name}: heads that lie end to end")


def _int32(x) -> int:
    """A bound as the C calls take it (ctypes would keep its low 32 bits)."""
    return min(int(x), 0x7fffffff)


_torch_parts = None


def _parts():
    """What calls on tensors need of torch, looked up once: int32, float32, the
    device guard, the current device's index (None where there is no other device
    that could be current) and the current stream's address by device index."""
    global _torch_parts
    if _torch_parts is None:
        import torch
        _torch_parts = (torch.int32, torch.float32, torch.cuda.device,
                        torch.cuda.current_device if torch.cuda.device_count() > 1 else None,
                        # without a Stream object for it
                        getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
                            lambda d: torch.cuda.current_stream(d).cuda_stream))
    return _torch_parts


class _OnDevice:
    """Calls on one device's tensors: its current stream, or a given one, with
    that device current."""

    def _place(self, device):
        self.device, self._dev = device, device.index
        self._i32, self._f32, self._guard, self._current, self._raw_stream = _parts()

    def _elsewhere(self, fn, *args) -> int:
        """fn(*args) with the tensors' device current, which it is not."""
        with self._guard(self._dev):
            return fn(*args)


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
        if axis_of_pair is None and sections is not None and len(sections) == 1:
            sections, half_of = None, sections[0]
            _need(half_of == half, "sections: rotary_dim / 2 pairs in all are wanted")
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
        axes = None if axis_of_pair is None else bytes(axis_of_pair)
        freq = None if inv_freq is None else (ctypes.c_double * half)(*[float(f) for f in inv_freq])
        _check(lib().mk_rope_init(ctypes.byref(self.c), rot, float(theta), freq, self.n_axes, axes),
               "mk_rope_init")
        self._p = ctypes.addressof(self.c)


class PagedBatch(_OnDevice):
    """The tables of a step (mk_paged_batch) over torch int32 CUDA tensors:
    block_table [n, max_blocks], cu_new [n + 1], kv_lens [n], and for build()
    and append positions and slots [max_tokens].  Holds references to them.
    `max_new`, the most new tokens of a request that attention expects (it selects
    the kernels: 1 for a decode step), may be set from step to step."""

    # Calls pass the structs by address without the interpreter's lock: one that a
    # call has is never written again, so that threads may share a batch.

    def __init__(self, block_table, cu_new, kv_lens, positions=None, slots=None, *, page_size: int,
                 max_new: int):
        lib()
        self._place(kv_lens.device)
        n = kv_lens.numel()
        _need(block_table.dim() == 2, "block_table: [n, max_blocks]")
        rows = None if slots is None else (slots.numel(),)
        _need((positions is None) == (slots is None), "positions and slots: both or neither")
        _tensors(self.device, kv_lens=(kv_lens, self._i32, (n,)), cu_new=(cu_new, self._i32, (n + 1,)),
                 block_table=(block_table, self._i32, (n, block_table.shape[1])),
                 slots=(slots, self._i32, rows), positions=(positions, self._i32, rows))
        self.block_table, self.cu_new, self.kv_lens = block_table, cu_new, kv_lens
        self.positions, self.slots = positions, slots
        self.n, self.page_size, self._max_new = n, page_size, _int32(max_new)
        self.max_tokens = 0 if slots is None else slots.numel()
        self.c = mk_paged_batch(_ptr(block_table), _ptr(cu_new), _ptr(kv_lens),
                                None if slots is None else _ptr(positions),
                                None if slots is None else _ptr(slots), n, block_table.shape[1],
                                self.max_tokens, self._max_new, page_size)
        self._p, self._build = ctypes.addressof(self.c), lib().mk_paged_tables
        self._rows = (self.max_tokens, self.c, self._p)

    @property
    def max_new(self) -> int:
        return self._max_new

    @max_new.setter
    def max_new(self, value: int) -> None:
        self._max_new = _int32(value)
        self._of_rows(self._rows[0])

    def _of_rows(self, rows: int):
        """(rows, struct with max_tokens = rows, its address) for attention; the
        last one asked for is kept."""
        c = mk_paged_batch.from_buffer_copy(self.c)
        c.max_tokens, c.max_new = rows, self._max_new
        self._rows = kept = (rows, c, ctypes.addressof(c))
        return kept

    def build(self, ctx_lens, new_lens, free_pages, n_free, n_left, status=None, stream=None) -> None:
        """mk_paged_tables: fill the tables from device int32 lengths [n], taking
        pages from the end of free_pages[0 : n_free[0]]; n_left[0] receives what
        remains.  `status` (int32 [1]) receives MK_ERR_BOUNDS where a request is
        refused.  No tensor that is written may be, or overlap, another of the
        call's (ctx_lens is not the batch's own kv_lens)."""
        i32, dev, n = self._i32, self._dev, self.n
        if not (ctx_lens.dtype is i32 and ctx_lens.get_device() == dev and ctx_lens.numel() == n
                and ctx_lens.is_contiguous() and new_lens.dtype is i32 and new_lens.get_device() == dev
                and new_lens.numel() == n and new_lens.is_contiguous() and free_pages.dtype is i32
                and free_pages.get_device() == dev and free_pages.is_contiguous() and n_free.dtype is i32
                and n_free.get_device() == dev and n_free.numel() == 1 and n_left.dtype is i32
                and n_left.get_device() == dev and n_left.numel() == 1 and self.slots is not None
                and (status is None or (status.dtype is i32 and status.get_device() == dev
                                        and status.numel() == 1))):
            _need(self.slots is not None, "build needs positions and slots")
            _tensors(self.device, ctx_lens=(ctx_lens, i32, (n,)), new_lens=(new_lens, i32, (n,)),
                     free_pages=(free_pages, i32, None), n_free=(n_free, i32, (1,)),
                     n_left=(n_left, i32, (1,)), status=(status, i32, (1,)))
        args = (self._p, ctx_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(),
                free_pages.numel(), n_free.data_ptr(), n_left.data_ptr(),
                None if status is None else status.data_ptr(),
                self._raw_stream(dev) if stream is None else int(stream.cuda_stream))
        if self._current is None or self._current() == dev:
            rc = self._build(*args)
        else:
            rc = self._elsewhere(self._build, *args)
        if rc:
            raise MkError(rc, "mk_paged_tables")


class PagedCache(_OnDevice):
    """One layer's paged cache (mk_paged_cache) over torch tensors k and v
    [n_pages, n_kv_heads, page_size, head_dim] of bf16 or fp16 (any view of that
    shape with contiguous head_dim, equal strides for both).  `workspace`
    (uint8, MK_PAGED_WORKSPACE_BYTES) may be shared by caches whose calls do not
    overlap; without one the first attention call allocates it.  Holds
    references to the tensors.  The status word is cleared on the stream that is
    current when the cache is made (outside of a capture); calls on other streams
    are ordered behind that by the caller, as behind one another.  A cache may be
    dropped while its calls run on any stream (its own memory, the status word and
    a workspace that it allocated, is then given back behind them); k, v and a given
    workspace are the caller's, and a captured graph needs the cache as long as it
    is replayed."""

    def __init__(self, k, v, n_q_heads: int, workspace=None):
        import torch
        _need(k.is_cuda and v.is_cuda and k.device == v.device and k.dtype == v.dtype
              and k.dtype in (torch.bfloat16, torch.float16), "k, v: CUDA tensors of bf16 or fp16")
        _need(k.dim() == 4 and k.shape == v.shape and k.stride() == v.stride() and k.stride(3) == 1,
              "k, v: [n_pages, n_kv_heads, page_size, head_dim], same strides")
        lib()
        self._place(k.device)
        n_pages, hkv, page, d = k.shape
        self.k, self.v, self.dtype = k, v, k.dtype
        self.n_q_heads, self.n_kv_heads, self.head_dim, self.page_size = n_q_heads, hkv, d, page
        self._status = torch.zeros(1, dtype=torch.int32, device=k.device)
        # streams on which the status word and an own workspace need no record (any more)
        self._home = self._raw_stream(self._dev)
        self.workspace, self._given, self._seen = None, workspace is not None, {self._home}
        s = k.stride()
        self.c = mk_paged_cache(_ptr(k), _ptr(v), None, _ptr(self._status), s[0], s[1], s[2],
                                n_q_heads, hkv, d, page, n_pages,
                                MK_BF16 if k.dtype == torch.bfloat16 else MK_FP16)
        self._p = ctypes.addressof(self.c)
        self._append, self._attention = lib().mk_paged_append, lib().mk_paged_attention
        if workspace is not None:
            _need(workspace.device == k.device and workspace.is_contiguous() and
                  workspace.numel() * workspace.element_size() >= MK_PAGED_WORKSPACE_BYTES,
                  "workspace: MK_PAGED_WORKSPACE_BYTES on the cache's device")
            self._set_workspace(workspace)

    def _first_on(self, stream, raw: int) -> None:
        """The first call on a stream that the cache's own memory is not of."""
        import torch
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        elif not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(raw, self.device)
        self._status.record_stream(stream)
        if self.workspace is not None and not self._given:
            self.workspace.record_stream(stream)
        self._seen.add(raw)

    def _set_workspace(self, t) -> None:
        self.workspace = t
        self.c.workspace = _ptr(t)

    def append(self, q, k, v, slots, positions=None, rope: Optional[Rope] = None, q_out=None,
               q_norm=None, k_norm=None, eps: float = 1e-6, stream=None) -> None:
        """mk_paged_append: q [T, n_q_heads, head_dim], k, v [T, n_kv_heads,
        head_dim], slots int32 [T], positions int32 [T] or [n_axes, T]; q_out
        defaults to q itself."""
        if q_out is None:
            q_out = q
        hq, hkv, d, dev, typ, i32 = self.n_q_heads, self.n_kv_heads, self.head_dim, self._dev, self.dtype, self._i32
        n = q.shape[0]
        qs, ks, vs, os = q.stride(), k.stride(), v.stride(), q_out.stride()
        wide, narrow = (n, hq, d), (n, hkv, d)
        if not (q.shape == wide and k.shape == narrow and v.shape == narrow
                and q.dtype is typ and k.dtype is typ and v.dtype is typ
                and q.get_device() == dev and k.get_device() == dev and v.get_device() == dev
                and (q_out is q or (q_out.shape == wide and q_out.dtype is typ and q_out.get_device() == dev))
                and qs[2] == ks[2] == vs[2] == os[2] == 1
                and (hq == 1 or qs[1] == os[1] == d) and (hkv == 1 or ks[1] == vs[1] == d)
                and slots.dtype is i32 and slots.get_device() == dev and slots.numel() == n
                and slots.is_contiguous()):
            _heads(self.device, typ, q=(q, wide), k=(k, narrow), v=(v, narrow), q_out=(q_out, wide))
            _tensors(self.device, slots=(slots, i32, (n,)))
        if (q_norm is not None or k_norm is not None):
            for g in (q_norm, k_norm):
                if g is not None and not (g.dtype is typ and g.get_device() == dev and g.shape == (d,)
                                          and g.is_contiguous()):
                    _tensors(self.device, q_norm=(q_norm, typ, (d,)), k_norm=(k_norm, typ, (d,)))
        pos, pos_stride, rp = None, 0, None
        if rope is not None:
            _need(positions is not None, "rope needs positions")
            shape, rp = positions.shape, rope._p
            if not (positions.dtype is i32 and positions.get_device() == dev and shape[-1] == n
                    and (shape == (rope.n_axes, n) or (len(shape) == 1 and rope.n_axes == 1))
                    and (n < 2 or positions.stride(-1) == 1)):
                raise ValueError(f"positions: int32 [{rope.n_axes}, {n}] on {self.device}, rows contiguous")
            pos = positions.data_ptr()
            if rope.n_axes > 1:
                pos_stride = positions.stride(0)
        if n == 0:
            return
        if n == 1:  # the stride of a lone token joins nothing and may be any number
            qs, ks, vs, os = (hq * d,), (hkv * d,), (hkv * d,), (hq * d,)
        raw = self._raw_stream(dev) if stream is None else int(stream.cuda_stream)
        if raw not in self._seen:
            self._first_on(stream, raw)
        args = (self._p, q.data_ptr(), qs[0], k.data_ptr(), ks[0], v.data_ptr(), vs[0], q_out.data_ptr(), os[0],
                None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(),
                eps, rp, pos, pos_stride, slots.data_ptr(), n, raw)
        if self._current is None or self._current() == dev:
            rc = self._append(*args)
        else:
            rc = self._elsewhere(self._append, *args)
        if rc:
            raise MkError(rc, "mk_paged_append")

    def attention(self, q, batch: PagedBatch, out, lse=None, scale: float = 0.0, window: int = 0,
                  stream=None) -> None:
        """mk_paged_attention: q, out [rows, n_q_heads, head_dim], lse float32
        [rows, n_q_heads] or None."""
        if self.workspace is None:
            import torch
            # on the call's stream: memory that another one has given back may
            # still be in use there
            with torch.cuda.device(self.device), torch.cuda.stream(stream):
                _need(not torch.cuda.is_current_stream_capturing(),
                      "workspace: give one, or call once before the capture (it would belong to the graph)")
                self._set_workspace(torch.empty(MK_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device=self.device))
            # (streams that have seen the status word alone have to see both)
            raw = self._raw_stream(self._dev) if stream is None else int(stream.cuda_stream)
            self._seen = {raw} if raw == self._home else set()
        hq, d, dev, typ = self.n_q_heads, self.head_dim, self._dev, self.dtype
        n = q.shape[0]
        wide, qs, os = (n, hq, d), q.stride(), out.stride()
        if not (q.shape == wide and out.shape == wide and q.dtype is typ and out.dtype is typ
                and q.get_device() == dev and out.get_device() == dev and batch._dev == dev
                and qs[2] == 1 and os[2] == 1 and (hq == 1 or (qs[1] == d and os[1] == d))
                and (lse is None or (lse.dtype is self._f32 and lse.get_device() == dev
                                     and lse.shape == (n, hq) and lse.is_contiguous()))):
            _heads(self.device, typ, q=(q, wide), out=(out, wide))
            _tensors(self.device, lse=(lse, self._f32, (n, hq)))
            _need(batch._dev == dev, "batch: on the cache's device")
        if n == 0:
            return
        if window > 0x7fffffff:  # past every position; ctypes would keep its low 32 bits
            window = 0
        rows = batch._rows  # held here until the call returns
        if rows[0] != n:
            rows = batch._of_rows(n)
        raw = self._raw_stream(dev) if stream is None else int(stream.cuda_stream)
        if raw not in self._seen:
            self._first_on(stream, raw)
        args = (self._p, rows[2], q.data_ptr(), qs[0] if n > 1 else hq * d, out.data_ptr(),
                os[0] if n > 1 else hq * d, None if lse is None else lse.data_ptr(), scale, window, raw)
        if self._current is None or self._current() == dev:
            rc = self._attention(*args)
        else:
            rc = self._elsewhere(self._attention, *args)
        if rc:
            raise MkError(rc, "mk_paged_attention")

    def status(self) -> int:
        """The status word: MK_OK or the first error latched by the cache's calls
        (waits for the current stream; calls on others have to be waited for)."""
        return int(self._status.item())

    def reset(self) -> None:
        self._status.zero_()
