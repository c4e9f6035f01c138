"""One decode step through the C ABI, with the buffers a caller keeps.

:class:`DecodeStep` owns what the runner page's ``T5DecodeRunner`` keeps
between steps (``__init__``: persistent, fixed-address plan buffers, the
partial/workspace area sized by slots, the packed-Q buffer and its
descales) and issues the four calls of a step: ``plan`` (host plan plus a
pinned, asynchronous copy into the fixed device buffers, mj_plan_upload), then
``mj_quantize_q``, ``mj_decode_attention`` and ``mj_merge_lse`` on one
stream. It holds no arithmetic of its own.
"""

from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

from . import (KV_FORMATS, LATENT_DIM, LATENT_ROPE_DIM, LATENT_ROW, MJ_IMPL_AUTO, MJ_KV_E2M1, MJ_KV_E4M3, MJ_OUT_BF16,
               MJ_OUT_F16, _check, _ptr, _same_device, _stream, load_library, mj_decode_args, mj_decode_attention,
               mj_latent_args, mj_latent_attention, mj_latent_plan, mj_latent_plan_size, mj_latent_slots,
               mj_latent_workspace_size, mj_latent_write_args, mj_merge_lse, mj_plan_split_kv, mj_plan_upload,
               mj_quantize_q, mj_rope_write_kv_args, mj_slots, mj_workspace_init, mj_workspace_size)


@dataclass
class PagedKV:
    """A paged K/V cache in device memory, as the decode call sees it."""

    k_cache: torch.Tensor  # uint8 buffer
    v_cache: torch.Tensor
    k_strides: tuple  # (page, token, head) in bytes
    v_strides: tuple
    page_size: int
    num_pages: int
    kv_format: str  # "fp8" | "e2m3" | "e3m2" | "e2m1"
    k_descale: torch.Tensor  # float32
    v_descale: torch.Tensor
    descale_strides: tuple  # (seq, head) in elements
    block_table: torch.Tensor  # int32 [B, max_blocks]
    seq_lens: torch.Tensor  # int32 [B]
    q_mul: torch.Tensor | None = None  # float32 [h_q, d]
    o_mul: torch.Tensor | None = None


class DecodeStep:
    def __init__(self, *, max_num_seqs: int, q_len: int, h_q: int, h_k: int, d: int = 128,
                 sm_count: int | None = None, ctas_per_sm: int = 2, max_splits: int = 16,
                 margin: int = 0, causal: bool = True, impl: int = MJ_IMPL_AUTO, kv_stages: int = 0,
                 evict_first: bool = True, device="cuda", with_lse: bool = False, q_mode: str = "fp8"):
        """``q_mode``: "fp8" (dynamic e4m3 Q, mj_quantize_q in the step),
        "fp8_fused" (the same quantization done by the decode kernel; the
        step is decode + merge) or "bf16" (Q as is; decode + merge)."""
        assert q_mode in ("fp8", "fp8_fused", "bf16")
        self.q_mode = q_mode
        self.device = torch.device(device)
        if sm_count is None:
            sm_count = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.max_num_seqs, self.q_len, self.h_q, self.h_k, self.d = max_num_seqs, q_len, h_q, h_k, d
        self.h_r = h_q // h_k
        self.n_q = q_len * self.h_r
        self.sm_count, self.ctas_per_sm, self.max_splits = sm_count, ctas_per_sm, max_splits
        self.margin, self.causal = margin, causal
        self.impl, self.kv_stages, self.evict_first = impl, kv_stages, evict_first
        self.slots = mj_slots(sm_count, ctas_per_sm, h_k, q_len, h_q)
        self.pad_to = max(self.slots, max_num_seqs)
        dev = self.device
        # fixed-address device plan buffers + pinned host staging
        self.work_dev = torch.zeros(self.pad_to, 4, dtype=torch.int32, device=dev)
        self.nsplit_dev = torch.ones(max(1, max_num_seqs), dtype=torch.int32, device=dev)
        self.work_host = torch.zeros(self.pad_to, 4, dtype=torch.int32).pin_memory()
        self.nsplit_host = torch.ones(max(1, max_num_seqs), dtype=torch.int32).pin_memory()
        self._staged = None  # event after the last H2D copy of the staging buffers
        # packed Q and its descales
        self.q_codes = torch.empty(max(1, max_num_seqs), h_k, self.n_q, d, dtype=torch.uint8, device=dev)
        self.q_descale = torch.ones(max(1, max_num_seqs), h_k, dtype=torch.float32, device=dev)
        # workspace: status word + partials sized by slots
        self.ws_bytes = mj_workspace_size(self.slots, max_splits, q_len, h_q, h_k, d)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        mj_workspace_init(self.workspace)
        self.lse = (torch.empty(max(1, max_num_seqs), h_k, self.n_q, dtype=torch.float32, device=dev)
                    if with_lse else None)
        self.plan_info = None

    # ------------------------------------------------------------------ plan
    def plan(self, seq_lens_host, num_seqs: int, stream=None) -> dict:
        """Host plan into the pinned staging buffers, then an asynchronous
        copy into the fixed device buffers on ``stream``."""
        if self._staged is not None:
            self._staged.synchronize()  # the previous copy has read the staging buffers
        info = mj_plan_split_kv(np.asarray(seq_lens_host, dtype=np.int32), num_seqs, self.q_len, self.h_q,
                                self.h_k, self.sm_count, self.ctas_per_sm, self.max_splits, self.margin,
                                self.pad_to, work_out=self.work_host, n_splits_out=self.nsplit_host)
        s = stream or torch.cuda.current_stream(self.device)
        mj_plan_upload(self.work_host, self.nsplit_host, self.work_dev, self.nsplit_dev, self.pad_to, num_seqs, s)
        if self._staged is None:
            self._staged = torch.cuda.Event()
        self._staged.record(s)
        info["num_seqs"] = num_seqs
        self.plan_info = info
        return info

    # ------------------------------------------------------------- the calls
    def args(self, kv: PagedKV, out: torch.Tensor, num_seqs: int, softmax_scale: float,
             q: torch.Tensor | None = None) -> mj_decode_args:
        """The decode call's arguments; ``q`` (bf16 mode): the bf16 Q it reads."""
        for name, t in (("out", out), ("q", q), ("k_cache", kv.k_cache), ("v_cache", kv.v_cache),
                        ("k_descale", kv.k_descale), ("v_descale", kv.v_descale), ("block_table", kv.block_table),
                        ("seq_lens", kv.seq_lens), ("q_mul", kv.q_mul), ("o_mul", kv.o_mul)):
            if t is not None and not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor: the kernels read it through a device pointer")
        info = self.plan_info
        a = mj_decode_args()
        if self.q_mode in ("bf16", "fp8_fused"):
            assert q is not None and q.dtype == torch.bfloat16 and q.stride(2) == 1
            a.q_mode, a.q_bf16 = (1 if self.q_mode == "bf16" else 2), q.data_ptr()
            a.q_tok_stride, a.q_head_stride = q.stride(0), q.stride(1)
            if self.q_mode == "fp8_fused" and kv.q_mul is not None:
                a.q_mul = kv.q_mul.data_ptr()
        a.num_seqs, a.q_len, a.h_q, a.h_k, a.d = num_seqs, self.q_len, self.h_q, self.h_k, self.d
        a.causal = 1 if self.causal else 0
        a.softmax_scale = softmax_scale
        a.q_codes, a.q_descale = self.q_codes.data_ptr(), self.q_descale.data_ptr()
        a.kv_format, a.page_size, a.num_pages = KV_FORMATS[kv.kv_format], kv.page_size, kv.num_pages
        a.k_cache, a.v_cache = kv.k_cache.data_ptr(), kv.v_cache.data_ptr()
        a.k_stride_page, a.k_stride_token, a.k_stride_head = kv.k_strides
        a.v_stride_page, a.v_stride_token, a.v_stride_head = kv.v_strides
        a.k_descale, a.v_descale = kv.k_descale.data_ptr(), kv.v_descale.data_ptr()
        a.descale_seq_stride, a.descale_head_stride = kv.descale_strides
        a.block_table, a.block_table_stride = kv.block_table.data_ptr(), kv.block_table.stride(0)
        a.seq_lens = kv.seq_lens.data_ptr()
        a.work, a.n_splits = self.work_dev.data_ptr(), self.nsplit_dev.data_ptr()
        a.num_work = self.pad_to
        a.with_reduction = 1 if info["with_reduction"] else 0
        a.chunk_tiles, a.max_splits, a.part_seqs = info["chunk_tiles"], self.max_splits, self.slots
        a.o_mul = kv.o_mul.data_ptr() if kv.o_mul is not None else None
        assert out.dtype in (torch.bfloat16, torch.float16), "the decode output is bf16 or fp16"
        a.out = out.data_ptr()
        a.out_dtype = 1 if out.dtype == torch.float16 else 0
        a.out_tok_stride, a.out_head_stride = out.stride(0), out.stride(1)
        a.lse = self.lse.data_ptr() if self.lse is not None else None
        a.workspace, a.workspace_bytes = self.workspace.data_ptr(), self.ws_bytes
        a.impl, a.kv_stages, a.evict_first = self.impl, self.kv_stages, 1 if self.evict_first else 0
        return a

    def run(self, q: torch.Tensor, out: torch.Tensor, kv: PagedKV, num_seqs: int, softmax_scale: float,
            stream=None, args: mj_decode_args | None = None):
        """Quantize Q (fp8 mode), decode, merge: the device part of one step."""
        if self.q_mode == "fp8":
            mj_quantize_q(q, num_seqs, self.q_len, self.h_k, self.q_codes, self.q_descale, q_mul=kv.q_mul,
                          stream=stream)
        a = args if args is not None else self.args(kv, out, num_seqs, softmax_scale, q=q)
        mj_decode_attention(a, stream)
        mj_merge_lse(a, stream)
        return out


def paged_kv_from_workload(w, device="cuda") -> PagedKV:
    """Move a synthetic workload's cache, tables and scales to the device."""
    dev = torch.device(device)
    k = torch.from_numpy(np.ascontiguousarray(w.k_cache)).to(dev)
    v = torch.from_numpy(np.ascontiguousarray(w.v_cache)).to(dev)
    ks = torch.from_numpy(np.ascontiguousarray(w.k_scale, dtype=np.float32)).to(dev)
    vs = torch.from_numpy(np.ascontiguousarray(w.v_scale, dtype=np.float32)).to(dev)
    ds = (0, 0) if w.k_scale.size == 1 else (0, 1)
    bt = torch.from_numpy(np.ascontiguousarray(w.block_table)).to(dev)
    sl = torch.from_numpy(np.ascontiguousarray(w.seq_lens)).to(dev)
    qm = torch.from_numpy(w.q_mul).to(dev) if w.q_mul is not None else None
    om = torch.from_numpy(w.o_mul).to(dev) if w.o_mul is not None else None
    return PagedKV(k_cache=k, v_cache=v, k_strides=tuple(w.kv_strides), v_strides=tuple(w.kv_strides),
                   page_size=w.page_size, num_pages=w.num_pages, kv_format=w.kv_format, k_descale=ks,
                   v_descale=vs, descale_strides=ds, block_table=bt, seq_lens=sl, q_mul=qm, o_mul=om)


def q_from_workload(w, device="cuda") -> torch.Tensor:
    return torch.from_numpy(w.q_bits.view(np.int16)).view(torch.bfloat16).to(device)


# ----------------------------------------------------------------------------
# the rotated cache writes
# ----------------------------------------------------------------------------
def _tensor(name: str, t: torch.Tensor, dtype, *shape) -> torch.Tensor:
    """Check a tensor the library reads through a device pointer: on a GPU, of
    the type, of the shape (None: any extent)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor: the kernels read it through a device pointer")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and int(n) != w for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple('*' if w is None else w for w in shape)}")
    return t


def _rows(name: str, t: torch.Tensor, dtype, *shape) -> torch.Tensor:
    _tensor(name, t, dtype, *shape)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: its last dimension must be contiguous")
    return t


def _flat(name: str, t: torch.Tensor, dtype, *shape) -> torch.Tensor:
    _tensor(name, t, dtype, *shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _pool(name: str, t: torch.Tensor, strides, page_size: int, num_pages: int, heads: int, row_bytes: int):
    """Check a cache that the library writes through a pointer and strides: on a
    GPU, uint8, and its last row ends inside the tensor."""
    if not t.is_cuda or t.dtype != torch.uint8:
        raise ValueError(f"{name} must be a uint8 CUDA tensor")
    page, token, head = strides
    need = (num_pages - 1) * page + (page_size - 1) * token + (heads - 1) * head + row_bytes if num_pages > 0 else 0
    have = 1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())) if t.numel() else 0
    if need > have:
        raise ValueError(f"{name}: {num_pages} pages of {page_size} tokens end at byte {need}, the tensor at {have}")


def _hold(a, *tensors):
    """``a`` keeps the tensors whose addresses it holds, and their one device."""
    held = [t for t in tensors if t is not None]
    devices = {t.device.index for t in held}
    if len(devices) > 1:
        raise ValueError(f"the tensors are on several devices: {sorted(devices)}")
    a.tensors, a.device_index = held, devices.pop()
    return a


def _set_rope(r, positions, turns, freq_axis, interleaved: bool, scale: float, T: int, d: int):
    axes = 1 if positions.dim() == 1 else int(positions.shape[0])
    if positions.dim() == 1:
        _flat("positions", positions, torch.int64, T)
    else:
        _rows("positions", positions, torch.int64, axes, T)
    n = int(turns.numel())
    _flat("turns", turns, torch.int64, n)
    if freq_axis is not None:
        _flat("freq_axis", freq_axis, torch.uint8, n)
    r.positions, r.axis_stride, r.num_axes = positions.data_ptr(), positions.stride(0) if axes > 1 else 0, axes
    r.turns, r.freq_axis = turns.data_ptr(), freq_axis.data_ptr() if freq_axis is not None else None
    r.rot_dim, r.interleaved, r.scale = 2 * n, 1 if interleaved else 0, float(scale)


def rope_write_args(q, key, value, positions, turns, slot_mapping, k_cache, v_cache, kv_strides, page_size: int,
                    num_pages: int, kv_format: int, k_scale, v_scale, *, q_out=None, freq_axis=None,
                    interleaved: bool = False, rope_scale: float = 1.0, scale_per_head: bool = False,
                    status=None) -> mj_rope_write_kv_args:
    """The arguments of :func:`mj_rope_write_kv`, good for as many calls as the
    buffers keep their addresses.

    ``q`` bf16 ``[T, h_q, d]`` or None (no queries) and ``q_out`` the same
    (None: in place); ``positions`` int64 ``[T]`` or ``[axes, T]``; ``turns``
    :func:`mj_rope_turns` of ``rot_dim / 2`` frequencies, on the device;
    ``freq_axis`` uint8, the axis of each frequency. The rest as for
    :func:`mj_write_kv`; the pages and strides must lie inside the caches."""
    T, h_k, d = (int(n) for n in key.shape)
    _rows("key", key, torch.bfloat16, T, h_k, d)
    _rows("value", value, torch.bfloat16, T, h_k, d)
    _flat("slot_mapping", slot_mapping, torch.int64, T)
    strides = tuple(int(x) for x in kv_strides)
    bits = {MJ_KV_E4M3: 8, MJ_KV_E2M1: 4}.get(int(kv_format), 6)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _pool(name, t, strides, int(page_size), int(num_pages), h_k, d * bits // 8)
    n_scale = h_k * d if kv_format != MJ_KV_E4M3 else (h_k if scale_per_head else 1)
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != n_scale:
            raise ValueError(f"{name}: {n_scale} contiguous float32 values on the GPU are required")
    a = mj_rope_write_kv_args()
    _set_rope(a.rope, positions, turns, freq_axis, interleaved, rope_scale, T, d)
    if q is not None:
        a.h_q = int(q.shape[1])
        _rows("q", q, torch.bfloat16, T, a.h_q, d)
        q_out = q if q_out is None else q_out
        _rows("q_out", q_out, torch.bfloat16, T, a.h_q, d)
        a.q, a.q_tok_stride, a.q_head_stride = q.data_ptr(), q.stride(0), q.stride(1)
        a.q_out, a.q_out_tok_stride, a.q_out_head_stride = q_out.data_ptr(), q_out.stride(0), q_out.stride(1)
    w = a.kv
    w.num_tokens, w.h_k, w.d = T, h_k, d
    w.key, w.key_tok_stride, w.key_head_stride = key.data_ptr(), key.stride(0), key.stride(1)
    w.value, w.value_tok_stride, w.value_head_stride = value.data_ptr(), value.stride(0), value.stride(1)
    w.slot_mapping = slot_mapping.data_ptr()
    w.kv_format, w.page_size, w.num_pages = int(kv_format), int(page_size), int(num_pages)
    w.k_cache, w.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
    w.k_stride_page, w.k_stride_token, w.k_stride_head = strides
    w.v_stride_page, w.v_stride_token, w.v_stride_head = strides
    w.k_scale, w.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
    w.scale_per_head = 1 if scale_per_head else 0
    w.status = _ptr(status)
    return _hold(a, q, q_out, key, value, positions, turns, freq_axis, slot_mapping, k_cache, v_cache, k_scale, v_scale,
                 status)


def _latent_cache(cache):
    _rows("cache", cache, torch.uint8, None, None, LATENT_ROW)
    return cache


def latent_write_args(q_pe, latent, k_pe, positions, turns, slot_mapping, cache, scale, *, q_out=None, freq_axis=None,
                      interleaved: bool = True, rope_scale: float = 1.0, status=None) -> mj_latent_write_args:
    """The arguments of :func:`mj_latent_write`, good for as many calls as the
    buffers keep their addresses.

    ``q_pe`` bf16 ``[T, h, 64]`` or None (no queries) and ``q_out`` the same
    (None: in place; usually the last 64 channels of the ``[T, h, 576]`` query);
    ``latent`` bf16 ``[T, 512]``, ``k_pe`` bf16 ``[T, 64]``; ``cache`` uint8
    ``[pages, page_size, 576]`` (any page and token strides); ``scale`` float32
    ``[2]`` (latent, key part). Positions as for :func:`rope_write_args`."""
    T = int(latent.shape[0])
    _rows("latent", latent, torch.bfloat16, T, LATENT_DIM)
    _rows("k_pe", k_pe, torch.bfloat16, T, LATENT_ROPE_DIM)
    _flat("slot_mapping", slot_mapping, torch.int64, T)
    _flat("scale", scale, torch.float32, 2)
    _latent_cache(cache)
    a = mj_latent_write_args()
    _set_rope(a.rope, positions, turns, freq_axis, interleaved, rope_scale, T, LATENT_ROPE_DIM)
    a.num_tokens = T
    if q_pe is not None:
        a.h = int(q_pe.shape[1])
        _rows("q_pe", q_pe, torch.bfloat16, T, a.h, LATENT_ROPE_DIM)
        q_out = q_pe if q_out is None else q_out
        _rows("q_out", q_out, torch.bfloat16, T, a.h, LATENT_ROPE_DIM)
        a.q_pe, a.q_tok_stride, a.q_head_stride = q_pe.data_ptr(), q_pe.stride(0), q_pe.stride(1)
        a.q_out, a.q_out_tok_stride, a.q_out_head_stride = q_out.data_ptr(), q_out.stride(0), q_out.stride(1)
    a.latent, a.latent_tok_stride = latent.data_ptr(), latent.stride(0)
    a.k_pe, a.k_pe_tok_stride = k_pe.data_ptr(), k_pe.stride(0)
    a.slot_mapping = slot_mapping.data_ptr()
    a.page_size, a.num_pages = int(cache.shape[1]), int(cache.shape[0])
    a.cache, a.stride_page, a.stride_token = cache.data_ptr(), cache.stride(0), cache.stride(1)
    a.scale = scale.data_ptr()
    a.status = _ptr(status)
    return _hold(a, q_pe, q_out, latent, k_pe, positions, turns, freq_axis, slot_mapping, cache, scale, status)


# ----------------------------------------------------------------------------
# attention over the latent cache
# ----------------------------------------------------------------------------
@dataclass
class PagedLatent:
    """A paged latent cache in device memory, as mj_latent_attention sees it."""

    cache: torch.Tensor  # uint8 [pages, page_size, 576]: e4m3 codes, any page and token strides
    descale: torch.Tensor  # float32 [2]: latent, key part
    block_table: torch.Tensor  # int32 [B, max_blocks]
    seq_lens: torch.Tensor  # int32 [B]; 0 = padding request


class LatentStep:
    """Latent attention with the buffers a caller keeps between steps: the plan
    (pinned staging and its fixed device buffer) and the workspace. One plan
    serves every layer of a step; calls that may run at once need a LatentStep
    each (they share its workspace)."""

    def __init__(self, *, max_num_seqs: int, q_len: int, h: int, sm_count: int | None = None, margin: int = 0,
                 causal: bool = True, evict_first: bool = True, device="cuda", with_lse: bool = False):
        self.device = torch.device(device)
        if sm_count is None:
            sm_count = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.max_num_seqs, self.q_len, self.h = max_num_seqs, q_len, h
        self.margin, self.causal, self.evict_first = margin, causal, evict_first
        self.slots = mj_latent_slots(sm_count, q_len, h)
        words = mj_latent_plan_size(self.slots, max_num_seqs)
        self.plan_dev = torch.zeros(words, dtype=torch.int32, device=self.device)
        self.plan_host = torch.zeros(words, dtype=torch.int32).pin_memory()
        self._staged = None  # event after the last copy of the staging buffer
        self.ws_bytes = mj_latent_workspace_size(self.slots, q_len, h)
        with torch.cuda.device(self.device):
            self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
            mj_workspace_init(self.workspace)
        self.lse = (torch.empty(max(1, max_num_seqs), q_len * h, dtype=torch.float32, device=self.device)
                    if with_lse else None)
        # the buffers may be used on any stream from here on: their clearing is done
        torch.cuda.current_stream(self.device).synchronize()

    def plan(self, seq_lens_host, num_seqs: int, stream=None):
        """Host plan into the pinned staging buffer, then an asynchronous copy
        into the fixed device buffer on ``stream``. The step's device must be the
        current one (a default stream is the current device's)."""
        _same_device("the step's buffers", self.plan_dev.device.index)
        if self._staged is not None:
            self._staged.synchronize()  # the previous copy has read the staging buffer
        mj_latent_plan(seq_lens_host, num_seqs, self.max_num_seqs, self.slots, self.q_len, self.h, self.margin,
                       plan_out=self.plan_host)
        s = stream or torch.cuda.current_stream(self.device)
        _check("mj_plan_upload", load_library().mj_plan_upload(
            self.plan_host.data_ptr(), None, self.plan_dev.data_ptr(), None, self.plan_host.numel() // 4, 0, _stream(s)))
        if self._staged is None:
            self._staged = torch.cuda.Event()
        self._staged.record(s)
        return self.plan_host

    def args(self, q: torch.Tensor, out: torch.Tensor, kv: PagedLatent, num_seqs: int,
             softmax_scale: float) -> mj_latent_args:
        """The attention call's arguments, good for as many calls as the
        buffers keep their addresses. ``q`` bf16 ``[>= num_seqs * q_len, h, 576]``,
        ``out`` bf16 or fp16 ``[>= num_seqs * q_len, h, 512]``."""
        if num_seqs > self.max_num_seqs:
            raise ValueError(f"{num_seqs} requests, the step was made for {self.max_num_seqs}")
        _rows("q", q, torch.bfloat16, None, self.h, LATENT_ROW)
        if out.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("out must be bf16 or fp16")
        _rows("out", out, out.dtype, None, self.h, LATENT_DIM)
        _latent_cache(kv.cache)
        _flat("descale", kv.descale, torch.float32, 2)
        _rows("block_table", kv.block_table, torch.int32, None, None)
        _flat("seq_lens", kv.seq_lens, torch.int32, None)
        if min(int(q.shape[0]), int(out.shape[0])) < num_seqs * self.q_len:
            raise ValueError(f"q and out need {num_seqs * self.q_len} rows")
        if min(int(kv.block_table.shape[0]), int(kv.seq_lens.shape[0])) < num_seqs:
            raise ValueError(f"block_table and seq_lens need {num_seqs} requests")
        a = mj_latent_args()
        a.num_seqs, a.max_num_seqs, a.q_len, a.h = num_seqs, self.max_num_seqs, self.q_len, self.h
        a.causal, a.softmax_scale = 1 if self.causal else 0, softmax_scale
        a.q, a.q_tok_stride, a.q_head_stride = q.data_ptr(), q.stride(0), q.stride(1)
        a.cache, a.stride_page, a.stride_token = kv.cache.data_ptr(), kv.cache.stride(0), kv.cache.stride(1)
        a.page_size, a.num_pages = int(kv.cache.shape[1]), int(kv.cache.shape[0])
        a.descale = kv.descale.data_ptr()
        a.block_table, a.block_table_stride = kv.block_table.data_ptr(), kv.block_table.stride(0)
        a.block_table_len = int(kv.block_table.shape[1])
        a.seq_lens, a.plan, a.slots = kv.seq_lens.data_ptr(), self.plan_dev.data_ptr(), self.slots
        a.out, a.out_tok_stride, a.out_head_stride = out.data_ptr(), out.stride(0), out.stride(1)
        a.out_dtype = MJ_OUT_F16 if out.dtype == torch.float16 else MJ_OUT_BF16
        a.lse = self.lse.data_ptr() if self.lse is not None else None
        a.workspace, a.workspace_bytes = self.workspace.data_ptr(), self.ws_bytes
        a.evict_first = 1 if self.evict_first else 0
        return _hold(a, q, out, kv.cache, kv.descale, kv.block_table, kv.seq_lens, self.plan_dev, self.workspace, self.lse)

    def run(self, q: torch.Tensor, out: torch.Tensor, kv: PagedLatent, num_seqs: int, softmax_scale: float, stream=None,
            args: mj_latent_args | None = None):
        """The device part of one layer's attention; ``plan`` comes before it."""
        mj_latent_attention(args if args is not None else self.args(q, out, kv, num_seqs, softmax_scale), stream)
        return out
