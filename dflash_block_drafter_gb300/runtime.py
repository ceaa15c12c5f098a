"""Device-memory plumbing around the libdflash C ABI, using PyTorch tensors.

PyTorch only allocates device memory and provides streams here; every step of
the draft pass runs in libdflash's CUDA kernels through the ctypes binding.
"""
from __future__ import annotations

from typing import Dict, Optional

import numpy as np
import torch

from . import (DFLASH_ERR_INVALID_ARG, DFLASH_MAX_BLOCK, DFLASH_T_BF16, DFLASH_T_FP16, DFLASH_T_FP32, DflashError,
               DflashKv4Cache, dflash_accept, dflash_commit_positions, dflash_draft_block, dflash_fuse_context,
               dflash_model_create, dflash_model_dequantize, dflash_model_destroy, dflash_model_device_bytes, dflash_state_create,
               dflash_state_destroy, dflash_state_device_bytes, dflash_state_read_kv, dflash_state_status,
               dflash_state_read_draft_probs, dflash_state_set_spec_min_p, dflash_state_write_kv, load_library,
               dflash_state_set_defer_kv, dflash_state_flush,
               dflash_kv4_attention, dflash_kv4_attention_workspace, dflash_kv4_bytes, dflash_kv4_read,
               dflash_kv4_prefix_attention, dflash_kv4_prefix_attention_workspace, dflash_kv4_write,
               dflash_page_tables, dflash_qk_norm_rope, dflash_rope_turns, dflash_sample_tokens, dflash_token_logprobs,
               make_config, make_weights)


def _stream(stream: Optional[torch.cuda.Stream] = None) -> int:
    return (stream or torch.cuda.current_stream()).cuda_stream


def to_device(arr: np.ndarray, device) -> torch.Tensor:
    """Copy a numpy array's bytes to the device (uint16 travels as int16)."""
    a = np.ascontiguousarray(arr)
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(a).to(device)


class DraftModel:
    """A libdflash model built from a checkpoint dict (numpy arrays of BF16
    bits / GGUF bytes, names as in include/dflash.h).  Keeps the borrowed
    embedding and LM head alive for the model's lifetime."""

    def __init__(self, cfg, ckpt: Dict[str, np.ndarray], device="cuda:0", keep_sources: bool = False):
        load_library()
        self.cfg = cfg
        self.device = torch.device(device)
        self.ccfg = make_config(cfg.n_layers, cfg.hidden, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim,
                                cfg.intermediate, cfg.vocab, cfg.n_taps, cfg.rope_theta, cfg.norm_eps,
                                cfg.mask_token_id, cfg.weight_type, getattr(cfg, "attn_window", 0))
        with torch.cuda.device(self.device):
            src = {k: to_device(v, self.device) for k, v in ckpt.items()}
            ptrs = {k: t.data_ptr() for k, t in src.items()}
            w = make_weights(ptrs, cfg.n_layers)
            self.handle = dflash_model_create(self.ccfg, w)
        # the target's embedding and LM head are borrowed, the rest was copied
        self.embed = src["embed"]
        self.head = src["head"]
        self.sources = src if keep_sources else None
        del src

    @property
    def device_bytes(self) -> int:
        return dflash_model_device_bytes(self.handle)

    def dequantize(self, which: int) -> torch.Tensor:
        cfg = self.cfg
        shapes = list(cfg.matrix_shapes().values())
        names = ["fc"] + [f"layers.{l}.{t}" for l in range(cfg.n_layers)
                          for t in ("wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down")]
        n, k = cfg.matrix_shapes()[names[which]]
        out = torch.empty((n, k), dtype=torch.float32, device=self.device)
        dflash_model_dequantize(self.handle, which, out.data_ptr(), _stream())
        return out

    def close(self):
        if getattr(self, "handle", None):
            dflash_model_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class DraftState:
    """A libdflash state (per-slot FP16 K/V + pass workspace) with
    preallocated device I/O buffers."""

    def __init__(self, model: DraftModel, n_slots: int, capacity: int):
        self.model = model
        self.n_slots = n_slots
        self.capacity = capacity
        dev = model.device
        with torch.cuda.device(dev):
            self.handle = dflash_state_create(model.handle, n_slots, capacity)
        cfg = model.cfg
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.drafts = torch.full((n_slots, DFLASH_MAX_BLOCK - 1), -7, dtype=torch.int32, device=dev)
        self.final_hidden = torch.zeros((n_slots, 8, cfg.hidden), dtype=torch.float32, device=dev)
        self.anchor_tok = torch.zeros(n_slots, dtype=torch.int32, device=dev)
        self.anchor_pos = torch.zeros(n_slots, dtype=torch.int32, device=dev)
        self.block_len = torch.zeros(n_slots, dtype=torch.int32, device=dev)

    @property
    def device_bytes(self) -> int:
        return dflash_state_device_bytes(self.handle)

    def fuse(self, slot: int, taps: torch.Tensor, positions: torch.Tensor, stream=None) -> None:
        assert taps.is_cuda and positions.is_cuda and positions.dtype == torch.int32
        n = positions.numel()
        dflash_fuse_context(self.model.handle, self.handle, slot, taps.data_ptr(), positions.data_ptr(), n,
                            self.status.data_ptr(), _stream(stream))
        # a deferring state reads the positions again in a later call: keep them alive
        self._kept_positions = positions if getattr(self, "_defer_kv", False) and n <= 8 else None

    def draft(self, n_seq: int, want_hidden: bool = True, stream=None) -> None:
        """Draft with the anchor_tok / anchor_pos / block_len buffers as set."""
        dflash_draft_block(self.model.handle, self.handle, n_seq, self.anchor_tok.data_ptr(),
                           self.anchor_pos.data_ptr(), self.block_len.data_ptr(), self.drafts.data_ptr(),
                           self.final_hidden.data_ptr() if want_hidden else 0, self.status.data_ptr(),
                           _stream(stream))

    def read_kv(self, slot: int, layer: int, pos0: int, n: int):
        cfg = self.model.cfg
        k = torch.empty((cfg.n_kv_heads, n, cfg.head_dim), dtype=torch.float32, device=self.model.device)
        v = torch.empty_like(k)
        dflash_state_read_kv(self.handle, slot, layer, pos0, n, k.data_ptr(), v.data_ptr(), _stream())
        return k, v

    def write_kv(self, slot: int, layer: int, pos0: int, k16: torch.Tensor, v16: torch.Tensor) -> None:
        """k16, v16: float16 / int16 tensors [n_kv, n, d] on the device."""
        n = k16.shape[1]
        dflash_state_write_kv(self.handle, slot, layer, pos0, n, k16.data_ptr(), v16.data_ptr(), _stream())

    def set_defer_kv(self, on: bool) -> None:
        """Leave the K/V of 8-position fusions to the next one-slot draft pass."""
        dflash_state_set_defer_kv(self.handle, on)
        self._defer_kv = bool(on)

    def flush(self, stream=None) -> None:
        """Project the K/V of rows a deferring fusion kept, now."""
        dflash_state_flush(self.handle, _stream(stream))

    def set_spec_min_p(self, floor: float) -> None:
        """Confidence floor of the offered drafts (0: all)."""
        dflash_state_set_spec_min_p(self.handle, floor)

    def draft_probs(self) -> torch.Tensor:
        """[n_slots, 7] float confidences of the last pass's drafts (-1: none)."""
        out = torch.empty((self.n_slots, DFLASH_MAX_BLOCK - 1), dtype=torch.float32, device=self.model.device)
        dflash_state_read_draft_probs(self.handle, out.data_ptr(), _stream())
        return out

    def take_status(self) -> int:
        torch.cuda.synchronize(self.model.device)
        v = int(self.status.item())
        self.status.zero_()
        return v

    def close(self):
        if getattr(self, "handle", None):
            dflash_state_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def accept(drafts: torch.Tensor, target_ids: torch.Tensor, block_len: torch.Tensor, accept_len: torch.Tensor,
           next_anchor: torch.Tensor, anchor_pos: Optional[torch.Tensor] = None, stream=None) -> None:
    n_seq, max_b = target_ids.shape
    dflash_accept(drafts.data_ptr(), target_ids.data_ptr(), block_len.data_ptr(), n_seq, max_b,
                  accept_len.data_ptr(), next_anchor.data_ptr(), anchor_pos.data_ptr() if anchor_pos is not None
                  else 0, _stream(stream))


def commit_positions(anchor_pos: torch.Tensor, accept_len: torch.Tensor, positions: torch.Tensor,
                     stream=None) -> None:
    """positions [n_seq, 8] <- the rows the next fusion commits (-1: none)."""
    dflash_commit_positions(anchor_pos.data_ptr(), accept_len.data_ptr(), accept_len.numel(),
                            positions.data_ptr(), _stream(stream))


# -------------------------------------------------------------- verify step
# The operators of include/dflash.h's verify step on torch tensors.  Each runs
# on the device of its tensors, on that device's current stream; with `stream`
# as if called inside torch.cuda.stream(stream), so that outputs and workspaces
# come from that stream's memory.  `status` is an optional int32 tensor for the
# DFLASH_DEV_* bits.
# (Small calls take as long as their Python: the checks are plain ones.)
_VALUE_TYPES = {torch.float32: DFLASH_T_FP32, torch.bfloat16: DFLASH_T_BF16, torch.float16: DFLASH_T_FP16}
_INT32 = torch.int32


def _refuse(what: str):
    raise DflashError(DFLASH_ERR_INVALID_ARG, what)


def _elsewhere(dev: torch.device, stream):
    """The context that makes the call's device and stream the current ones; None if they are."""
    if stream is not None:
        if stream.device_index != dev.index:
            _refuse("the stream is of another device")
        return torch.cuda.stream(stream)
    return torch.cuda.device(dev) if dev.index != torch.cuda.current_device() else None


def _current(dev: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _int32(device, what: str, *tensors) -> None:
    for x in tensors:
        if x is not None and (x.dtype != _INT32 or x.device != device or not x.is_contiguous()):
            _refuse(what + ": contiguous int32 tensors on the device of the call")


def kv4_cache(n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, device="cuda:0") -> torch.Tensor:
    """A zeroed 4-bit paged K/V cache: uint8 [n_pages, n_kv_heads, page_size / 16, 18 * head_dim]."""
    load_library()
    if dflash_kv4_bytes(n_pages, page_size, n_kv_heads, head_dim) == 0:
        _refuse("kv4_cache: geometry")
    return torch.zeros((n_pages, n_kv_heads, page_size // 16, 18 * head_dim), dtype=torch.uint8, device=device)


def _kv4(cache: torch.Tensor) -> DflashKv4Cache:
    if not (cache.is_cuda and cache.dtype == torch.uint8 and cache.dim() == 4 and cache.is_contiguous()):
        _refuse("a 4-bit cache is a contiguous uint8 tensor of kv4_cache's shape")
    n_pages, heads, groups, size = cache.shape
    if size % 18:
        _refuse("a 4-bit cache is a contiguous uint8 tensor of kv4_cache's shape")
    return DflashKv4Cache(cache.data_ptr(), n_pages, 16 * groups, heads, size // 18)


def _row_stride(x: torch.Tensor, device, what: str) -> int:
    """Elements between the rows of [rows, heads, head_dim] values whose heads are dense."""
    if x.dim() != 3 or x.device != device or x.dtype not in _VALUE_TYPES:
        _refuse(what + ": [rows, heads, head_dim] values on the device of the call")
    rows, heads, d = x.shape
    stride, by_head, by_value = x.stride()
    if by_value != 1 or (by_head != d and heads > 1):
        _refuse(what + ": the heads of a row must be dense")
    return stride if rows > 1 else heads * d


def page_tables(lengths: torch.Tensor, new_rows: torch.Tensor, held: torch.Tensor, table: torch.Tensor,
                ring: torch.Tensor, ring_state: torch.Tensor, page_size: int, row_cap: int, held_out=None,
                ring_state_out=None, status=None, stream=None):
    """Take and give back pages for requests that append rows; returns
    (row_offsets [n_seq + 1], slots [row_cap], positions [row_cap]).  `table`
    and `ring` are updated in place, `held` and `ring_state` too unless
    held_out / ring_state_out are given."""
    dev = table.device
    if not table.is_cuda:
        _refuse("page_tables: CUDA tensors")
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return page_tables(lengths, new_rows, held, table, ring, ring_state, page_size, row_cap, held_out,
                               ring_state_out, status)
    if held_out is None:
        held_out = held
    if ring_state_out is None:
        ring_state_out = ring_state
    _int32(dev, "page_tables", lengths, new_rows, held, table, ring, ring_state, held_out, ring_state_out, status)
    n = lengths.numel()
    if (table.dim() != 2 or table.shape[0] != n or new_rows.numel() != n or held.numel() != n or held_out.numel() != n
            or ring_state.numel() != 2 or ring_state_out.numel() != 2 or row_cap < 0):
        _refuse("page_tables: sizes")
    wide = (row_cap + 3) & ~3  # slots and positions start on 16 bytes
    out = torch.empty(2 * wide + n + 1, dtype=_INT32, device=dev)
    at = out.data_ptr()
    dflash_page_tables(lengths.data_ptr(), new_rows.data_ptr(), n, page_size, ring.numel(), held.data_ptr(),
                       held_out.data_ptr(), table.data_ptr(), table.shape[1], ring.data_ptr(), ring_state.data_ptr(),
                       ring_state_out.data_ptr(), at + 8 * wide, at, at + 4 * wide, row_cap,
                       0 if status is None else status.data_ptr(), _current(dev))
    return out[2 * wide:], out[:row_cap], out[wide: wide + row_cap]


def kv4_write(cache: torch.Tensor, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, status=None,
              stream=None) -> None:
    """Quantise rows k, v [n, n_kv_heads, head_dim] into the cells `slots` [n] (-1: none)."""
    c, dev = _kv4(cache), cache.device
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return kv4_write(cache, k, v, slots, status)
    ks, vs = _row_stride(k, dev, "kv4_write k"), _row_stride(v, dev, "kv4_write v")
    _int32(dev, "kv4_write slots", slots, status)
    n, heads, d = k.shape
    if k.shape != v.shape or k.dtype != v.dtype or n != slots.numel() or heads != c.n_kv_heads or d != c.head_dim:
        _refuse("kv4_write: shapes")
    dflash_kv4_write(c, k.data_ptr(), v.data_ptr(), _VALUE_TYPES[k.dtype], ks, vs, slots.data_ptr(), n,
                     0 if status is None else status.data_ptr(), _current(dev))


def kv4_read(cache: torch.Tensor, slots: torch.Tensor, status=None, stream=None):
    """(k, v), float [n, n_kv_heads, head_dim], of the cells `slots` (zeros for -1)."""
    c, dev = _kv4(cache), cache.device
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return kv4_read(cache, slots, status)
    _int32(dev, "kv4_read slots", slots, status)
    n = slots.numel()
    k = torch.empty((n, c.n_kv_heads, c.head_dim), dtype=torch.float32, device=dev)
    v = torch.empty((n, c.n_kv_heads, c.head_dim), dtype=torch.float32, device=dev)
    dflash_kv4_read(c, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), 0 if status is None else status.data_ptr(),
                    _current(dev))
    return k, v


def kv4_attention(cache: torch.Tensor, q: torch.Tensor, table: torch.Tensor, kv_len: torch.Tensor,
                  row_offsets: torch.Tensor, max_rows: int, causal: bool = True, window: int = 0,
                  scale: Optional[float] = None, out=None, workspace=None, status=None, stream=None) -> torch.Tensor:
    """Attention of rows q [tokens, n_q_heads, head_dim] over the cells of
    their sequences; scale None is head_dim ** -0.5.  Rows of no sequence keep
    what `out` held (unset if out is None)."""
    c, dev = _kv4(cache), cache.device
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return kv4_attention(cache, q, table, kv_len, row_offsets, max_rows, causal, window, scale, out, workspace,
                                 status)
    qs = _row_stride(q, dev, "kv4_attention q")
    _int32(dev, "kv4_attention", table, kv_len, row_offsets, status)
    tokens, heads, d = q.shape
    n = kv_len.numel()
    if d != c.head_dim or table.dim() != 2 or table.shape[0] != n or row_offsets.numel() != n + 1:
        _refuse("kv4_attention: shapes")
    if out is None:
        out, os_ = torch.empty((tokens, heads, d), dtype=q.dtype, device=dev), heads * d
    else:
        if out.shape != q.shape or out.dtype != q.dtype:
            _refuse("kv4_attention: out")
        os_ = _row_stride(out, dev, "kv4_attention out")
    if workspace is None:
        size = dflash_kv4_attention_workspace(c, heads, n, max_rows, table.shape[1])
        workspace = torch.empty(size + 16, dtype=torch.uint8, device=dev)
    else:
        size = workspace.numel() * workspace.element_size()
        if workspace.device != dev or not workspace.is_contiguous():
            _refuse("kv4_attention: workspace")
    dflash_kv4_attention(c, q.data_ptr(), out.data_ptr(), _VALUE_TYPES[q.dtype], qs, os_, tokens, heads, n, max_rows,
                         row_offsets.data_ptr(), kv_len.data_ptr(), table.data_ptr(), table.shape[1], causal, window,
                         d ** -0.5 if scale is None else scale, workspace.data_ptr(), size,
                         0 if status is None else status.data_ptr(), _current(dev))
    return out


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, top_k: int = 0, status=None,
                   stream=None):
    """Scores of logits [rows, vocab]: (logprob [rows] of `tokens` or None,
    entropy [rows], top_ids [rows, top_k], top_logprobs [rows, top_k])."""
    dev = logits.device
    kind = _VALUE_TYPES.get(logits.dtype)
    if not logits.is_cuda or logits.dim() != 2 or kind is None:
        _refuse("token_logprobs: [rows, vocab] logits on a CUDA device")
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return token_logprobs(logits, tokens, top_k, status)
    n, vocab = logits.shape
    stride, by_value = logits.stride()
    if (by_value != 1 and vocab != 1) or (tokens is not None and tokens.numel() != n) or top_k < 0:
        _refuse("token_logprobs: dense rows, one token each")
    _int32(dev, "token_logprobs", tokens, status)
    logp = None if tokens is None else torch.empty(n, dtype=torch.float32, device=dev)
    entropy = torch.empty(n, dtype=torch.float32, device=dev)
    ids = torch.empty((n, top_k), dtype=_INT32, device=dev)
    top = torch.empty((n, top_k), dtype=torch.float32, device=dev)
    dflash_token_logprobs(logits.data_ptr(), kind, stride if n > 1 else vocab, n, vocab,
                          0 if tokens is None else tokens.data_ptr(), 0 if logp is None else logp.data_ptr(),
                          entropy.data_ptr(), top_k, ids.data_ptr(), top.data_ptr(),
                          0 if status is None else status.data_ptr(), _current(dev))
    return logp, entropy, ids, top


# ------------------------------------------------------------ sampling step
# (as the verify step's: each on the device of its tensors, on its current stream or on `stream`)
def rope_turns(inv_freq, device="cuda:0") -> torch.Tensor:
    """The rotation table of qk_norm_rope: int64 [rotary_dim / 2] (the bits of
    unsigned integers) of frequencies in radians per position."""
    turns = np.array(dflash_rope_turns(inv_freq), dtype=np.uint64).view(np.int64)
    return torch.from_numpy(turns).to(device)


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                 turns: Optional[torch.Tensor], q_weight=None, k_weight=None, eps: float = 1e-6, axes=None, q_out=None,
                 k_out=None, status=None, stream=None):
    """Per-head norm (with q_weight / k_weight, float [head_dim]) and rotation
    of rows q [n, n_q_heads, head_dim] and k [n, n_k_heads, head_dim] (or None) at
    `positions` [n], or [n_axes, n] with `axes` (uint8, one per frequency).
    Returns (q_out, k_out), which may be q and k themselves; rows of a negative
    position keep what they held (unset if the outputs are made here)."""
    dev, dtype = q.device, q.dtype
    if not q.is_cuda:
        _refuse("qk_norm_rope: CUDA tensors")
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return qk_norm_rope(q, k, positions, turns, q_weight, k_weight, eps, axes, q_out, k_out, status)
    qs = _row_stride(q, dev, "qk_norm_rope q")
    n, heads, d = q.shape
    if q_out is None:
        q_out, qos = torch.empty((n, heads, d), dtype=dtype, device=dev), heads * d
    else:
        qos = _row_stride(q_out, dev, "qk_norm_rope q_out")
        if q_out.shape != q.shape or q_out.dtype != dtype:
            _refuse("qk_norm_rope q_out: the rows' shape and type")
    kp = kop = None
    ks = kos = k_heads = 0
    if k is not None:
        ks = _row_stride(k, dev, "qk_norm_rope k")
        kn, k_heads, kd = k.shape
        if kn != n or kd != d or k.dtype != dtype:
            _refuse("qk_norm_rope: rows of one length and type")
        if k_out is None:
            k_out, kos = torch.empty((n, k_heads, d), dtype=dtype, device=dev), k_heads * d
        else:
            kos = _row_stride(k_out, dev, "qk_norm_rope k_out")
            if k_out.shape != k.shape or k_out.dtype != dtype:
                _refuse("qk_norm_rope k_out: the rows' shape and type")
        kp, kop = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None or k_weight is not None:
        _refuse("qk_norm_rope: k_out and k_weight without k")
    qw = kw = None
    if q_weight is not None:
        qw = _weight(q_weight, dev, d)
    if k_weight is not None:
        kw = _weight(k_weight, dev, d)
    half, n_axes, pos, tp, ap = 0, 1, None, None, None
    if turns is not None:
        half = turns.numel()
        if positions is None or turns.dtype != torch.int64 or turns.device != dev or not turns.is_contiguous():
            _refuse("qk_norm_rope: positions, and contiguous int64 turns on the device of the call")
        if positions.dim() == 2:
            n_axes = positions.shape[0]
        if positions.numel() != n_axes * n or positions.dim() > 2:
            _refuse("qk_norm_rope: positions [n] or [n_axes, n]")
        if n_axes > 1 and axes is None:
            _refuse("qk_norm_rope: several axes need `axes`")
        if axes is not None:
            if axes.dtype != torch.uint8 or axes.device != dev or axes.numel() != half or not axes.is_contiguous():
                _refuse("qk_norm_rope: axes are contiguous uint8, one per frequency")
            ap = axes.data_ptr()
        _int32(dev, "qk_norm_rope", positions, status)
        pos, tp = positions.data_ptr(), turns.data_ptr()
    elif status is not None:
        _int32(dev, "qk_norm_rope", status)
    dflash_qk_norm_rope(q.data_ptr(), q_out.data_ptr(), qs, qos, heads, kp, kop, ks, kos, k_heads, d,
                        _VALUE_TYPES[dtype], n, qw, kw, eps, pos, n, n_axes, ap, tp, 2 * half,
                        None if status is None else status.data_ptr(), _current(dev))
    return q_out, k_out


def _weight(w: torch.Tensor, device, d: int) -> int:
    if w.dtype != torch.float32 or w.device != device or w.numel() != d or not w.is_contiguous():
        _refuse("qk_norm_rope: weights are contiguous float [head_dim] on the device of the call")
    return w.data_ptr()


def kv4_prefix_attention(cache: torch.Tensor, q: torch.Tensor, prefix_table: torch.Tensor, prefix_len: torch.Tensor,
                         group_offsets: torch.Tensor, table: torch.Tensor, kv_len: torch.Tensor,
                         row_offsets: torch.Tensor, max_rows: int, causal: bool = True, scale: Optional[float] = None,
                         out=None, workspace=None, status=None, stream=None) -> torch.Tensor:
    """Attention of rows q [tokens, n_q_heads, head_dim] over the prefix that
    their group of sequences shares and the cells of their own sequence, which
    `table` and `kv_len` describe; else as kv4_attention."""
    c, dev = _kv4(cache), cache.device
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return kv4_prefix_attention(cache, q, prefix_table, prefix_len, group_offsets, table, kv_len, row_offsets,
                                        max_rows, causal, scale, out, workspace, status)
    qs = _row_stride(q, dev, "kv4_prefix_attention q")
    _int32(dev, "kv4_prefix_attention", prefix_table, prefix_len, group_offsets, table, kv_len, row_offsets, status)
    tokens, heads, d = q.shape
    n, groups = kv_len.numel(), prefix_len.numel()
    if (d != c.head_dim or table.dim() != 2 or table.shape[0] != n or row_offsets.numel() != n + 1
            or prefix_table.dim() != 2 or prefix_table.shape[0] != groups or group_offsets.numel() != groups + 1):
        _refuse("kv4_prefix_attention: shapes")
    if out is None:
        out, os_ = torch.empty((tokens, heads, d), dtype=q.dtype, device=dev), heads * d
    else:
        if out.shape != q.shape or out.dtype != q.dtype:
            _refuse("kv4_prefix_attention: out")
        os_ = _row_stride(out, dev, "kv4_prefix_attention out")
    if workspace is None:
        size = dflash_kv4_prefix_attention_workspace(c, tokens, heads, groups, prefix_table.shape[1], n, max_rows,
                                                     table.shape[1])
        workspace = torch.empty(size + 16, dtype=torch.uint8, device=dev)
    else:
        size = workspace.numel() * workspace.element_size()
        if workspace.device != dev or not workspace.is_contiguous():
            _refuse("kv4_prefix_attention: workspace")
    dflash_kv4_prefix_attention(c, q.data_ptr(), out.data_ptr(), _VALUE_TYPES[q.dtype], qs, os_, tokens, heads, groups,
                                group_offsets.data_ptr(), prefix_len.data_ptr(), prefix_table.data_ptr(),
                                prefix_table.shape[1], n, max_rows, row_offsets.data_ptr(), kv_len.data_ptr(),
                                table.data_ptr(), table.shape[1], causal, d ** -0.5 if scale is None else scale,
                                workspace.data_ptr(), size, 0 if status is None else status.data_ptr(), _current(dev))
    return out


def sample_tokens(logits: torch.Tensor, uniform: torch.Tensor, temperature=None, top_k=None, top_p=None, min_p=None,
                  status=None, stream=None):
    """Draw a token from each row of logits [rows, vocab] by the numbers
    `uniform` [rows] in [0, 1): (tokens [rows], logprob [rows] among the kept
    tokens, kept [rows]).  temperature, top_p, min_p (float) and top_k (int32)
    are [rows] tensors on the device, or None (off)."""
    dev = logits.device
    kind = _VALUE_TYPES.get(logits.dtype)
    if not logits.is_cuda or logits.dim() != 2 or kind is None:
        _refuse("sample_tokens: [rows, vocab] logits on a CUDA device")
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return sample_tokens(logits, uniform, temperature, top_k, top_p, min_p, status)
    n, vocab = logits.shape
    stride, by_value = logits.stride()
    if by_value != 1 and vocab != 1:
        _refuse("sample_tokens: dense rows")
    if top_k is not None or status is not None:
        _int32(dev, "sample_tokens", top_k, status)
        if top_k is not None and top_k.numel() != n:
            _refuse("sample_tokens: one top_k per row")
    out = torch.empty((3, n), dtype=_INT32, device=dev)
    to = out.data_ptr()
    dflash_sample_tokens(logits.data_ptr(), kind, stride if n > 1 else vocab, n, vocab, _of_row(uniform, dev, n),
                         _of_row(temperature, dev, n), None if top_k is None else top_k.data_ptr(),
                         _of_row(top_p, dev, n), _of_row(min_p, dev, n), to, to + 4 * n, to + 8 * n,
                         None if status is None else status.data_ptr(), _current(dev))
    tokens, logprob, kept = out.unbind()
    return tokens, logprob.view(torch.float32), kept


def _of_row(x: Optional[torch.Tensor], device, n: int) -> Optional[int]:
    if x is None:
        return None
    if x.dtype != torch.float32 or x.device != device or x.numel() != n or not x.is_contiguous():
        _refuse("sample_tokens: one contiguous float of the device of the call per row")
    return x.data_ptr()
