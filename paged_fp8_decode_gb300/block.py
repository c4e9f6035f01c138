"""The block-scaled cache through the C ABI: its arguments' checks, and the
buffers a caller keeps between steps.

The cache holds e4m3 codes and, for each block of tokens and KV head, one
exponent byte ``e``: a code ``c`` stands for ``c * 2^(e - 127)``. The exponents are
found as tokens are written (:func:`block_write_args`), so the cache needs no
calibrated scales. :class:`BlockStep` is decode attention over it,
:class:`PromptStep` attention of prompt chunks, :func:`block_read_args` brings
tokens back as rows.
"""

from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (MJ_OUT_BF16, MJ_OUT_F16, _check, _same_device, _stream, load_library, mj_block_args, mj_block_attention,
               mj_block_cache, mj_block_plan, mj_block_plan_size, mj_block_prompt, mj_block_prompt_args,
               mj_block_prompt_splits, mj_block_prompt_workspace_size, mj_block_read_args, mj_block_slots,
               mj_block_workspace_size, mj_block_write_args, mj_workspace_init)
from .step import _flat, _hold, _rows, _tensor


@dataclass
class BlockKV:
    """A block-scaled cache in device memory. Pages, tokens and heads may lie in
    any order (views of another layout); attention wants K and V alike in whether
    a token's heads or a head's tokens lie closer together. ``k_exp`` and ``v_exp``
    have a column for each block of a page, which sets the block: page_size / columns
    tokens."""

    k_cache: torch.Tensor  # uint8 [pages, page_size, h_k, d]: e4m3 codes, channels contiguous
    v_cache: torch.Tensor
    k_exp: torch.Tensor  # uint8 [pages, h_k, page_size / block], blocks contiguous
    v_exp: torch.Tensor

    @staticmethod
    def empty(num_pages: int, page_size: int, h_k: int, d: int, block: int, device="cuda") -> "BlockKV":
        """A cache of zeros, each page's heads apart (a head's tokens are contiguous)."""
        def pool():
            return torch.zeros(num_pages, h_k, page_size, d, dtype=torch.uint8, device=device).transpose(1, 2)

        def exps():
            return torch.full((num_pages, h_k, page_size // block), 127, dtype=torch.uint8, device=device)

        return BlockKV(pool(), pool(), exps(), exps())


def _set_cache(c: mj_block_cache, kv: BlockKV):
    _rows("k_cache", kv.k_cache, torch.uint8, None, None, None, None)
    pages, page_size, h_k, d = (int(n) for n in kv.k_cache.shape)
    _rows("v_cache", kv.v_cache, torch.uint8, pages, page_size, h_k, d)
    _rows("k_exp", kv.k_exp, torch.uint8, pages, h_k, None)
    blocks = int(kv.k_exp.shape[2])
    _rows("v_exp", kv.v_exp, torch.uint8, pages, h_k, blocks)
    if blocks < 1 or page_size % blocks:
        raise ValueError(f"a page of {page_size} tokens does not hold {blocks} blocks")
    c.h_k, c.d, c.page_size, c.block, c.num_pages = h_k, d, page_size, page_size // blocks, pages
    c.k_cache, c.v_cache = kv.k_cache.data_ptr(), kv.v_cache.data_ptr()
    c.k_stride_page, c.k_stride_token, c.k_stride_head = kv.k_cache.stride()[:3]
    c.v_stride_page, c.v_stride_token, c.v_stride_head = kv.v_cache.stride()[:3]
    c.k_exp, c.v_exp = kv.k_exp.data_ptr(), kv.v_exp.data_ptr()
    c.k_exp_stride_page, c.k_exp_stride_head = kv.k_exp.stride()[:2]
    c.v_exp_stride_page, c.v_exp_stride_head = kv.v_exp.stride()[:2]
    return h_k, d


def _status(status):
    return None if status is None else _flat("status", status, torch.int32, 1).data_ptr()


def _held(kv: BlockKV):
    return kv.k_cache, kv.v_cache, kv.k_exp, kv.v_exp


def block_write_args(key, value, slot_mapping, kv: BlockKV, *, status=None) -> mj_block_write_args:
    """The arguments of :func:`mj_block_write_kv`, good for as many calls as the
    buffers keep their addresses. ``key``, ``value`` bf16 ``[T, h_k, d]`` (any token
    and head strides); ``slot_mapping`` int64 ``[T]``, negative = padding; the
    tokens of one block follow one another; ``status`` an optional int32 word."""
    a = mj_block_write_args()
    h_k, d = _set_cache(a.cache, kv)
    T = int(key.shape[0])
    _rows("key", key, torch.bfloat16, T, h_k, d)
    _rows("value", value, torch.bfloat16, T, h_k, d)
    _flat("slot_mapping", slot_mapping, torch.int64, T)
    a.num_tokens, a.key, a.value, a.slot_mapping = T, key.data_ptr(), value.data_ptr(), slot_mapping.data_ptr()
    a.key_tok_stride, a.key_head_stride = key.stride()[:2]
    a.value_tok_stride, a.value_head_stride = value.stride()[:2]
    a.status = _status(status)
    return _hold(a, key, value, slot_mapping, *_held(kv), status)


def _set_table(a, block_table, num_seqs: int):
    _rows("block_table", block_table, torch.int32, None, None)
    if int(block_table.shape[0]) < num_seqs:
        raise ValueError(f"block_table needs {num_seqs} requests")
    a.block_table, a.block_table_stride, a.block_table_len = block_table.data_ptr(), block_table.stride(0), block_table.shape[1]


def block_read_args(kv: BlockKV, block_table, starts, k_out=None, v_out=None, *, first=None,
                    status=None) -> mj_block_read_args:
    """The arguments of :func:`mj_block_read_kv`. ``starts`` int32 ``[num_seqs + 1]``,
    the outputs' first row of each request; ``first`` int32 ``[num_seqs]``, the first
    token of each (None: 0); ``k_out``, ``v_out`` bf16 or fp16 ``[rows, h_k, d]`` (any
    token and head strides), either may be None."""
    a = mj_block_read_args()
    h_k, d = _set_cache(a.cache, kv)
    outs = [t for t in (k_out, v_out) if t is not None]
    if not outs:
        raise ValueError("neither k_out nor v_out is given")
    rows, dtype = int(outs[0].shape[0]), outs[0].dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("the outputs must be bf16 or fp16")
    _tensor("starts", starts, torch.int32, None)
    a.num_seqs, a.num_rows = int(starts.shape[0]) - 1, rows
    _flat("starts", starts, torch.int32, a.num_seqs + 1)
    if first is not None:
        _flat("first", first, torch.int32, a.num_seqs)
    _set_table(a, block_table, a.num_seqs)
    for name, t in (("k", k_out), ("v", v_out)):
        if t is not None:
            _rows(name + "_out", t, dtype, rows, h_k, d)
            setattr(a, name + "_out", t.data_ptr())
            setattr(a, name + "_tok_stride", t.stride(0))
            setattr(a, name + "_head_stride", t.stride(1))
    a.starts, a.first = starts.data_ptr(), first.data_ptr() if first is not None else None
    a.out_dtype = MJ_OUT_F16 if dtype == torch.float16 else MJ_OUT_BF16
    a.status = _status(status)
    return _hold(a, block_table, starts, first, k_out, v_out, *_held(kv), status)


def _set_io(a, q, out, h_q: int, d: int):
    if out.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("out must be bf16 or fp16")
    _rows("q", q, torch.bfloat16, None, h_q, d)
    _rows("out", out, out.dtype, None, h_q, d)
    a.q, a.q_tok_stride, a.q_head_stride = q.data_ptr(), q.stride(0), q.stride(1)
    a.out, a.out_tok_stride, a.out_head_stride = out.data_ptr(), out.stride(0), out.stride(1)
    a.out_dtype = MJ_OUT_F16 if out.dtype == torch.float16 else MJ_OUT_BF16


def _workspace(n: int, device):
    with torch.cuda.device(device):
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        mj_workspace_init(ws)
    return ws


class BlockStep:
    """Decode attention over a block-scaled cache with the buffers a caller keeps
    between steps: the plan (pinned staging and its fixed device buffer) and the
    workspace. One plan serves every layer of a step; calls that may run at once
    need a BlockStep each (they share its workspace). Make it for about as many requests
    as run: a call's grid has room for ``max_num_seqs`` (40 ragged requests of up to 16384
    tokens, 32/8 heads: 100 us made for 40, 130 for 1024; with 4 query tokens 136 and 170)."""

    def __init__(self, *, max_num_seqs: int, q_len: int, h_q: int, h_k: int, d: int, sm_count: int | None = None,
                 margin: int = 0, causal: bool = True, evict_first: bool = True, device="cuda",
                 with_lse: bool = False):
        self.device = torch.device(device)
        if sm_count is None:
            sm_count = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.max_num_seqs, self.q_len, self.h_q, self.h_k, self.d = max_num_seqs, q_len, h_q, h_k, d
        self.margin, self.causal, self.evict_first = margin, causal, evict_first
        self.slots = mj_block_slots(sm_count, q_len, h_q, h_k, d)
        words = mj_block_plan_size(self.slots, max_num_seqs)
        self.plan_dev = torch.zeros(words, dtype=torch.int32, device=self.device)
        self.plan_host = torch.zeros(words, dtype=torch.int32).pin_memory()
        self._staged = None  # event after the last copy of the staging buffer
        self.ws_bytes = mj_block_workspace_size(self.slots, q_len, h_q, h_k, d)
        self.workspace = _workspace(self.ws_bytes, self.device)
        self.lse = (torch.empty(max(1, max_num_seqs), h_k, q_len * (h_q // h_k), dtype=torch.float32, device=self.device)
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
        mj_block_plan(seq_lens_host, num_seqs, self.max_num_seqs, self.slots, self.margin, plan_out=self.plan_host)
        s = stream or torch.cuda.current_stream(self.device)
        _check("mj_plan_upload", load_library().mj_plan_upload(
            self.plan_host.data_ptr(), None, self.plan_dev.data_ptr(), None, self.plan_host.numel() // 4, 0, _stream(s)))
        if self._staged is None:
            self._staged = torch.cuda.Event()
        self._staged.record(s)
        return self.plan_host

    def args(self, q: torch.Tensor, out: torch.Tensor, kv: BlockKV, block_table, seq_lens, num_seqs: int,
             softmax_scale: float) -> mj_block_args:
        """The attention call's arguments, good for as many calls and plans as the
        buffers keep their addresses. ``q`` bf16 and ``out`` bf16 or fp16
        ``[>= num_seqs * q_len, h_q, d]``; ``block_table`` int32 ``[>= num_seqs, pages a
        request]``; ``seq_lens`` int32, 0 = padding request."""
        if num_seqs > self.max_num_seqs:
            raise ValueError(f"{num_seqs} requests, the step was made for {self.max_num_seqs}")
        a = mj_block_args()
        if _set_cache(a.cache, kv) != (self.h_k, self.d):
            raise ValueError(f"the step was made for {self.h_k} KV heads of {self.d} channels")
        _set_io(a, q, out, self.h_q, self.d)
        if min(int(q.shape[0]), int(out.shape[0])) < num_seqs * self.q_len:
            raise ValueError(f"q and out need {num_seqs * self.q_len} rows")
        _set_table(a, block_table, num_seqs)
        _flat("seq_lens", seq_lens, torch.int32, None)
        if int(seq_lens.shape[0]) < num_seqs:
            raise ValueError(f"seq_lens needs {num_seqs} requests")
        a.num_seqs, a.max_num_seqs, a.q_len, a.h_q = num_seqs, self.max_num_seqs, self.q_len, self.h_q
        a.causal, a.softmax_scale = 1 if self.causal else 0, softmax_scale
        a.seq_lens, a.plan, a.slots = seq_lens.data_ptr(), self.plan_dev.data_ptr(), self.slots
        a.lse = self.lse.data_ptr() if self.lse is not None else None
        a.workspace, a.workspace_bytes = self.workspace.data_ptr(), self.ws_bytes
        a.evict_first = 1 if self.evict_first else 0
        return _hold(a, q, out, block_table, seq_lens, self.plan_dev, self.workspace, self.lse, *_held(kv))

    def run(self, q, out, kv: BlockKV, block_table, seq_lens, num_seqs: int, softmax_scale: float, stream=None,
            args: mj_block_args | None = None):
        """The device part of one layer's attention; ``plan`` comes before it."""
        mj_block_attention(args if args is not None else self.args(q, out, kv, block_table, seq_lens, num_seqs,
                                                                   softmax_scale), stream)
        return out


class PromptStep:
    """Attention of ragged prompt chunks over a block-scaled cache, with the
    workspace a caller keeps. Calls that may run at once need a PromptStep each.

    ``max_tokens`` bounds the query tokens of a call, ``max_q_len`` those of one
    request, ``max_len`` a request's length; ``splits`` into how many pieces the keys
    are cut (None: as many as fill the GPU with the largest batch).

    The bounds also choose the kernel, the grid and the pieces of every call: make a
    step of their own for short or few chunks. (32/8 heads of 128, through a step for 64
    chunks of up to 4096 tokens, and through one for the chunks' own number and length: 64 tokens after 2000 36
    and 20 us, after 16000 196 and 32; 64 chunks of 20 tokens after 500 each 122 and 51; of 128 tokens 242 and 84.)"""

    def __init__(self, *, max_tokens: int, max_num_seqs: int, max_q_len: int, max_len: int, h_q: int, h_k: int, d: int,
                 sm_count: int | None = None, splits: int | None = None, causal: bool = True, device="cuda",
                 with_lse: bool = False):
        self.device = torch.device(device)
        if sm_count is None:
            sm_count = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.max_tokens, self.max_num_seqs, self.max_q_len = max_tokens, max_num_seqs, max_q_len
        self.h_q, self.h_k, self.d, self.causal = h_q, h_k, d, causal
        self.splits = splits if splits is not None else mj_block_prompt_splits(sm_count, max_num_seqs, max_q_len, max_len,
                                                                               h_q, h_k, d)
        self.ws_bytes = mj_block_prompt_workspace_size(max_tokens, h_q, d, self.splits)
        self.workspace = _workspace(self.ws_bytes, self.device)
        self.lse = torch.empty(max(1, max_tokens), h_q, dtype=torch.float32, device=self.device) if with_lse else None
        # the buffers may be used on any stream from here on: their clearing is done
        torch.cuda.current_stream(self.device).synchronize()

    def args(self, q: torch.Tensor, out: torch.Tensor, kv: BlockKV, block_table, seq_lens, q_starts, num_seqs: int,
             softmax_scale: float) -> mj_block_prompt_args:
        """The call's arguments, good for as many calls as the buffers keep their
        addresses. ``q`` bf16 and ``out`` bf16 or fp16 ``[T, h_q, d]``; ``q_starts`` int32
        ``[num_seqs + 1]``, the first row of each request's chunk; ``seq_lens`` int32, the
        requests' lengths with the chunk; the rest as for :meth:`BlockStep.args`."""
        T = int(q.shape[0])
        if T > self.max_tokens or num_seqs > self.max_num_seqs:
            raise ValueError(f"{T} query tokens of {num_seqs} requests, the step was made for {self.max_tokens} of "
                             f"{self.max_num_seqs}")
        a = mj_block_prompt_args()
        if _set_cache(a.cache, kv) != (self.h_k, self.d):
            raise ValueError(f"the step was made for {self.h_k} KV heads of {self.d} channels")
        _set_io(a, q, out, self.h_q, self.d)
        if int(out.shape[0]) < T:
            raise ValueError(f"out needs {T} rows")
        _set_table(a, block_table, num_seqs)
        _flat("seq_lens", seq_lens, torch.int32, None)
        _flat("q_starts", q_starts, torch.int32, None)
        if int(seq_lens.shape[0]) < num_seqs or int(q_starts.shape[0]) < num_seqs + 1:
            raise ValueError(f"seq_lens needs {num_seqs} requests, q_starts one more")
        a.num_seqs, a.num_tokens, a.max_q_len, a.splits = num_seqs, T, self.max_q_len, self.splits
        a.h_q, a.causal, a.softmax_scale = self.h_q, 1 if self.causal else 0, softmax_scale
        a.q_starts, a.seq_lens = q_starts.data_ptr(), seq_lens.data_ptr()
        a.lse = self.lse.data_ptr() if self.lse is not None else None
        a.workspace, a.workspace_bytes = self.workspace.data_ptr(), self.ws_bytes
        return _hold(a, q, out, block_table, seq_lens, q_starts, self.workspace, self.lse, *_held(kv))

    def run(self, q, out, kv: BlockKV, block_table, seq_lens, q_starts, num_seqs: int, softmax_scale: float, stream=None,
            args: mj_block_prompt_args | None = None):
        """One layer's attention of the chunks."""
        mj_block_prompt(args if args is not None else self.args(q, out, kv, block_table, seq_lens, q_starts, num_seqs,
                                                                softmax_scale), stream)
        return out
