"""4-bit pages in plain numpy: the quantiser by its definition, and fp64 attention over what the
pages hold.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares no code with the CUDA path.
bf16 arrays are uint16 bit patterns.  Codes are uint8 [pages, P, Hkv, D / 2] (byte j: dim 2 j in the
low four bits, 2 j + 1 in the high ones), or [pages, Hkv, P, D / 2] with layout "hnd"; parameters
uint16 [pages, Hkv, P, D / 64, 2] (scale, minimum of each group of 64 values).
"""
from __future__ import annotations

import math

import numpy as np

GROUP = 64
NAN_BITS = 0x7FC0


def bf16_value(bits) -> np.ndarray:
    """The fp32 values of bf16 bit patterns."""
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32)


def bf16_round(x) -> np.ndarray:
    """Bit patterns of finite fp32 values rounded to the nearest bf16 (ties to even)."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def quantise(bits):
    """bf16 bits [..., D] -> (codes uint8 [..., D / 2], params uint16 [..., D / 64, 2])."""
    x = bf16_value(bits)
    x = x.reshape(*x.shape[:-1], -1, GROUP)
    finite = np.isfinite(x).all(-1, keepdims=True)
    x = np.where(finite, x, np.float32(0))
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    half = np.float32(0.5)
    scale_bits = bf16_round((hi * half - lo * half) / np.float32(7.5))
    scale = bf16_value(scale_bits)
    ok = finite & (scale > 0)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        steps = np.rint((x * half - lo * half) / (np.where(ok, scale, np.float32(1)) * half))
    codes = np.where(ok, np.clip(steps, 0, 15), 0).astype(np.uint8)
    codes = codes.reshape(*codes.shape[:-2], -1)
    lo_bits = (np.ascontiguousarray(lo).view(np.uint32) >> 16).astype(np.uint16)
    params = np.concatenate([scale_bits, lo_bits], -1)
    params = np.where(finite, params, np.uint16(NAN_BITS))
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8), params


def values(codes, params) -> np.ndarray:
    """The fp64 values that codes [..., D / 2] with params [..., D / 64, 2] stand for."""
    u = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1, GROUP)
    p = bf16_value(params).astype(np.float64)
    v = p[..., 0:1] * u + p[..., 1:2]
    return v.reshape(*v.shape[:-2], -1)


def _rows(pool, layout):
    """The code pool as [pages, P, Hkv, D / 2], a view."""
    return pool if layout == "nhd" else pool.transpose(0, 2, 1, 3)


def store(k_codes, v_codes, k_params, v_params, k_new, v_new, slots, layout="nhd") -> None:
    """In place; slots below 0 are skipped."""
    slots = np.asarray(slots, dtype=np.int64)
    P = _rows(k_codes, layout).shape[1]
    live = slots >= 0
    page, off = slots[live] // P, slots[live] % P
    for codes, params, new in ((k_codes, k_params, k_new), (v_codes, v_params, v_new)):
        c, p = quantise(new[live])
        _rows(codes, layout)[page, off] = c
        params.transpose(0, 2, 1, 3, 4)[page, off] = p


def load(codes, params, slots, layout="nhd") -> np.ndarray:
    """fp64 [T, Hkv, D] of the slots; zeros where a slot is negative."""
    slots = np.asarray(slots, dtype=np.int64)
    rows = _rows(codes, layout)
    P = rows.shape[1]
    s = np.maximum(slots, 0)
    v = values(rows[s // P, s % P], params.transpose(0, 2, 1, 3, 4)[s // P, s % P])
    v[slots < 0] = 0.0
    return v


def attention(q, k_codes, v_codes, k_params, v_params, block_table, context_lens, scale=None,
              layout="nhd") -> np.ndarray:
    """fp64 [S, Hq, D]: one query per sequence over its positions; rows of 0 without any."""
    S, Hq, D = q.shape
    P, H = _rows(k_codes, layout).shape[1:3]
    G = Hq // H
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    out = np.zeros((S, Hq, D))
    for s in range(S):
        n = int(context_lens[s])
        if n == 0:
            continue
        p = np.arange(n)
        slots = block_table[s][p // P].astype(np.int64) * P + p % P
        k, v = load(k_codes, k_params, slots, layout), load(v_codes, v_params, slots, layout)
        qs = bf16_value(q[s]).astype(np.float64).reshape(H, G, D)
        x = np.einsum("hgd,lhd->hgl", qs, k) * scale
        x -= x.max(-1, keepdims=True)
        w = np.exp(x)
        w /= w.sum(-1, keepdims=True)
        out[s] = np.einsum("hgl,lhd->hgd", w, v).reshape(Hq, D)
    return out
