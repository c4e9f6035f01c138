"""The block-scaled cache (oracle side), in float64.

Test infrastructure only (see :mod:`oracle`). The pages have static scales; the
cache defined here finds its own:

* e4m3 codes, and for each block of tokens and KV head an exponent byte ``e``: a
  code ``c`` stands for ``c * 2^(e - 127)``, ``e`` held to 95 .. 159;
* a write sets ``e`` to the smallest with ``max |x| <= 448 * 2^(e - 127)`` over its
  finite values in the block, and not below the block's own unless it writes the
  block's first row; the rows before its first one move to the larger scale.
"""

from __future__ import annotations

import numpy as np

from .formats import e4m3_decode, e4m3_encode

BIAS, LOW, HIGH = 127, 95, 159


def need(amax: float) -> int:
    """The smallest exponent byte whose scale holds ``amax``."""
    e = LOW
    while e < HIGH and amax > 448.0 * 2.0 ** (e - BIAS):
        e += 1
    return e


def write(x, slots, codes, exps):
    """x float64 [T, h, d] (values of bf16 inputs) into copies of codes uint8
    [pages, page, h, d] and exps uint8 [pages, h, blocks]; returns both."""
    codes, exps = codes.copy(), exps.copy()
    pages, page, h, _ = codes.shape
    block = page // exps.shape[2]
    groups: dict = {}
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            groups.setdefault(int(s) // block, []).append((int(s) % block, t))
    for blk, rows in groups.items():
        pg, at = blk * block // page, blk * block % page
        first = min(r for r, _ in rows)
        for g in range(h):
            v = np.abs(x[[t for _, t in rows], g])
            e = need(float(v[np.isfinite(v)].max(initial=0.0)))
            old = min(max(int(exps[pg, g, at // block]), LOW), HIGH)
            if first > 0 and old < e:
                codes[pg, at:at + first, g] = e4m3_encode(e4m3_decode(codes[pg, at:at + first, g]) * 2.0 ** (old - e))
            if first > 0:
                e = max(e, old)
            exps[pg, g, at // block] = e
            for r, t in rows:
                codes[pg, at + r, g] = e4m3_encode(x[t, g] * 2.0 ** (BIAS - e))
    return codes, exps


def values(codes, exps):
    """float64 [pages, page, h, d]: what the codes stand for."""
    block = codes.shape[1] // exps.shape[2]
    e = np.clip(exps.astype(np.int64), LOW, HIGH) - BIAS
    return e4m3_decode(codes).astype(np.float64) * np.repeat(2.0 ** e, block, axis=2).transpose(0, 2, 1)[..., None]


def gather(vals, table_row, n):
    """[n, h, d]: a request's first n tokens."""
    at = np.arange(n)
    page = vals.shape[1]
    return vals[np.asarray(table_row)[at // page], at % page]


def attention(q, k, v, softmax_scale, causal):
    """One request: q [m, h_q, d], the last m of n tokens; k, v [n, h_k, d], all
    float64. Returns (out [m, h_q, d], lse [m, h_q]); a row that sees no key is 0
    with LSE -inf."""
    m, h_q, d = q.shape
    n, h_k, _ = k.shape
    r = h_q // h_k
    out, lse = np.zeros((m, h_q, d)), np.full((m, h_q), -np.inf)
    for g in range(h_k):
        logit = np.einsum("thd,nd->thn", q[:, g * r:(g + 1) * r], k[:, g]) * softmax_scale
        if causal:
            hidden = np.arange(n)[None] > (np.arange(m) + n - m)[:, None]
            logit = np.where(hidden[:, None], -np.inf, logit)
        top = logit.max(axis=2, initial=-np.inf, keepdims=True)
        w = np.exp(logit - np.where(np.isneginf(top), 0.0, top))
        total = w.sum(axis=2, keepdims=True)
        safe = np.where(total == 0, 1.0, total)
        out[:, g * r:(g + 1) * r] = np.einsum("thn,nd->thd", w / safe, v[:, g])
        with np.errstate(divide="ignore"):
            lse[:, g * r:(g + 1) * r] = (np.where(np.isneginf(top), 0.0, top) + np.log(total))[..., 0]
    return out, lse
