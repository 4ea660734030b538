"""Plain FP64 forms of the operators beside the expert forward, written from the definitions in
include/nvfp4moe.h with numpy; used by their tests only."""
from __future__ import annotations

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_values(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_round(v: np.ndarray) -> np.ndarray:
    """BF16 bits of FP64 values of normal magnitude, to nearest even in one rounding: an FP64 number has 45 fraction
    bits more than a BF16 one, whose bits are the top of it once the exponent is rebased."""
    u = np.asarray(v, np.float64).view(np.uint64).copy()
    u += np.uint64((1 << 44) - 1) + ((u >> np.uint64(45)) & np.uint64(1))
    exact = ((u >> np.uint64(45)) << np.uint64(45)).view(np.float64)
    return (exact.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


# --- expert selection -------------------------------------------------------------------------------

def usable_logits(logits):
    """(usable, clean logits) in FP64."""
    l = np.asarray(logits, np.float64)
    usable = ~np.isnan(l) & (l != -np.inf)
    return usable, np.where(usable, np.minimum(l, FLT_MAX), -np.inf)


def scores(l, usable, sigmoid):
    with np.errstate(over="ignore"):
        if sigmoid:
            return np.where(usable, 1.0 / (1.0 + np.exp(-np.where(usable, l, 0.0))), 0.0)
    if not usable.any():
        return np.zeros_like(l)
    e = np.where(usable, np.exp(np.where(usable, l - l[usable].max(), 0.0)), 0.0)
    return e / e.sum()


def weights(l, live, sigmoid, renorm, s):
    """Weights before the scale of the chosen experts with logits l and scores s."""
    if not renorm:
        return np.where(live, s, 0.0)
    if not live.any():
        return np.zeros_like(l)
    if sigmoid:
        logw = np.where(live, np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(np.where(live, l, 0.0)))), -np.inf)
    else:
        logw = np.where(live, l, -np.inf)
    w = np.exp(logw - logw.max())
    return w / w.sum()


def select_row(logits, k, bias=None, sigmoid=False, renorm=True, scale=1.0, n_groups=1, top_groups=1, top2=False):
    """(ids, probs) of one token."""
    usable, l = usable_logits(logits)
    s = scores(l, usable, sigmoid)
    b = np.zeros_like(l) if bias is None else np.asarray(bias, np.float64)
    live = usable & ~np.isnan(b) & (b != -np.inf)
    b = np.minimum(b, FLT_MAX)
    v = l if bias is None else s + b
    E = len(l)
    size = E // n_groups
    value = []
    for g in range(n_groups):
        best = sorted(((s + b) if top2 else v)[e] for e in range(g * size, (g + 1) * size) if live[e])[::-1]
        value.append(-np.inf if not best else sum(best[:2]) if top2 else best[0])
    kept = sorted(range(n_groups), key=lambda g: (-value[g], g))[:top_groups]
    able = [e for g in sorted(kept) for e in range(g * size, (g + 1) * size)]
    order = sorted(able, key=lambda e: (not live[e], -v[e] if live[e] else 0.0, e))[:k]
    ids = np.array(order)
    return ids, scale * weights(l[ids], live[ids], sigmoid, renorm, s[ids])


def select_backward_row(logits, ids, dprobs, bias=None, sigmoid=False, renorm=True, scale=1.0):
    usable, l = usable_logits(logits)
    E = len(l)
    s = scores(l, usable, sigmoid)
    inside = (ids >= 0) & (ids < E)
    at = np.where(inside, ids, 0)
    live = inside & usable[at]
    if bias is not None:
        b = np.asarray(bias, np.float64)[at]
        live &= ~np.isnan(b) & (b != -np.inf)
    w = weights(np.where(live, l[at], -np.inf), live, sigmoid, renorm, s[at])
    dp = np.asarray(dprobs, np.float64)
    mean = (w * dp)[live].sum()
    d = np.where(live, w * (dp - mean if renorm else dp), 0.0)
    if sigmoid:
        d = d * (1.0 - s[at])
    out = np.zeros(E)
    for j in range(len(ids)):
        if live[j]:
            out[ids[j]] += d[j]
    if not renorm and not sigmoid:
        out -= s * mean
    return scale * out


# --- MXFP4 --------------------------------------------------------------------------------------------

def mxfp4_quantize(bits, up):
    """BF16 bits [rows, cols] -> (4-bit codes [rows, cols], scale bytes [rows, cols / 32]): the scale searched among
    the powers of two, each code by its distance."""
    x = bf16_values(bits)
    rows, cols = x.shape
    blocks = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(blocks).all(2)
    m = np.abs(np.where(np.isfinite(blocks), blocks, 0.0)).max(2)
    k = np.full(m.shape, -127)
    for j in range(-127, 127):  # FLOOR: the largest k with 4 * 2^k <= m; RU: the smallest k with m <= 6 * 2^k
        k = np.where((6.0 * 2.0 ** (j - 1) < m) if up else (4.0 * 2.0 ** j <= m), j, k)
    q = np.abs(np.where(np.isfinite(blocks), blocks, 0.0)) / np.exp2(k.astype(np.float64))[..., None]
    dist = np.abs(q[..., None] - E2M1) + 1e-9 * (np.arange(8) % 2) * (q[..., None] < 6)  # ties to the even code
    code = dist.argmin(-1) | (np.signbit(blocks).astype(int) << 3)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(rows, cols), np.where(bad, 255, k + 127)


def mxfp4_values(code, byte):
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127.0))
    return (v.reshape(*byte.shape, 32) * s[..., None]).reshape(code.shape)


def mxfp4_tile_maps(rows, cols):
    """Byte offsets of the GEMM layout, from the header: code bytes [rows, cols / 2], scale bytes [rows, cols / 32]."""
    C, Q = -(-cols // 128), -(-(-(-cols // 128)) // 4)
    r = np.arange(rows)[:, None]
    k = np.arange(0, cols, 2)[None, :]
    code = ((r // 16) * C + k // 128) * 1024 + (k % 128 // 32 * 16 + r % 16) * 16 + (k % 32) // 2
    k = np.arange(0, cols, 32)[None, :]
    scale = ((r // 16) * Q + k // 128 // 4) * 256 + (k % 128 // 32 * 16 + r % 16) * 4 + k // 128 % 4
    return code, scale
