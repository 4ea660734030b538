"""Plain FP64 forms of the balance loss, the low-rank adapters and their gradients, from the definitions in
include/nvfp4moe.h with torch, and the error bounds of the kernels' sums; used by their tests only."""
from __future__ import annotations

import torch

FLT_MAX = float(torch.finfo(torch.float32).max)
U = 2.0 ** -24  # half a step of FP32, relative
BF16 = 2.0 ** -8  # of BF16


# --- balance loss -----------------------------------------------------------------------------------

def probabilities(logits, sigmoid):
    """(p, sigma) [T, E] over the usable logits; zeros in a row without one."""
    l = logits.double()
    usable = ~torch.isnan(l) & (l != -torch.inf)
    l = torch.where(usable, l.clamp(max=FLT_MAX), 0.0)
    if sigmoid:  # in logarithms, so that nothing vanishes
        logw = torch.where(usable, torch.nn.functional.logsigmoid(l), -torch.inf)
    else:
        logw = torch.where(usable, l, -torch.inf)
    top = logw.max(1, keepdim=True)[0]
    w = torch.where(usable, torch.exp(logw - torch.where(torch.isfinite(top), top, 0.0)), 0.0)
    return w / w.sum(1, keepdim=True).clamp(min=1e-300), torch.sigmoid(l)


def sequence_of(T, offsets, device):
    """(sequence of each row or -1, sequences)"""
    if offsets is None:
        return torch.zeros(T, dtype=torch.long, device=device), 1
    seq = torch.full((T,), -1, dtype=torch.long, device=device)
    off = [min(max(o, 0), T) for o in offsets.tolist()]
    for s, (a, b) in enumerate(zip(off, off[1:])):
        seq[a:b] = s
    return seq, len(off) - 1


def balance_loss(logits, ids, coef, sigmoid, offsets=None):
    T, E = logits.shape
    seq, S = sequence_of(T, offsets, logits.device)
    counts = torch.zeros(S, E, dtype=torch.int64, device=logits.device)
    p, _ = probabilities(logits, sigmoid)
    total, tokens = 0.0, int((seq >= 0).sum())
    for s in range(S):
        at = seq == s
        rows = int(at.sum())
        if rows == 0:
            continue
        i = ids[at].flatten().long()
        counts[s] = torch.bincount(i[(i >= 0) & (i < E)], minlength=E)
        f = counts[s].double() * E / (ids.shape[1] * rows)
        total += float((f * p[at].sum(0)).sum())
    return coef * total / max(tokens, 1), counts


def balance_backward(logits, counts, k, coef, sigmoid, offsets=None, dloss=1.0, add=None):
    """(gradient, bound of the kernel's error before the last rounding)"""
    T, E = logits.shape
    seq, S = sequence_of(T, offsets, logits.device)
    p, sig = probabilities(logits, sigmoid)
    rows = torch.stack([(seq == s).sum() for s in range(S)]).double()
    at = seq.clamp(min=0)
    c = torch.where(seq >= 0, dloss * coef * E / (k * max(float((seq >= 0).sum()), 1.0)) / rows[at].clamp(min=1), 0.0)[:, None]
    n = counts.double()[at]
    other = 1 - sig if sigmoid else torch.ones_like(sig)
    if sigmoid:  # where sigma is next to 1
        l = logits.double().nan_to_num(0.0, FLT_MAX, -FLT_MAX)
        other = torch.sigmoid(-l)
    # n_e - sum_j p_j n_j as sum_j p_j (n_e - n_j), in which nothing cancels where one p is next to 1
    diff = torch.stack([(p * (n[:, e:e + 1] - n)).sum(1) for e in range(E)], 1)
    spread = torch.stack([(p * (n[:, e:e + 1] - n).abs()).sum(1) for e in range(E)], 1)
    d = c * p * other * diff
    # w within 12 u (exponential, reciprocal, product), so D^2 within 24, n D - G = sum_j w_j (n_e - n_j) within 12 of
    # its terms; and D and G are FP64 sums of at most 22 rounded additions and 22 rounded products: 2^-53 * 23 each,
    # below 2^-48 of n_e D and of G, which is more where the difference itself is smaller than that
    bound = (c * p * other).abs() * (U * (50 * diff.abs() + 12 * spread) + 2.0 ** -48 * (n + (n * p).sum(1, keepdim=True))) + 1e-36
    if add is not None:
        d = d + add.double()
    return d, bound


# --- adapters ---------------------------------------------------------------------------------------

def chain(n):
    """Relative bound of an FP32 sum by the matrix instructions: 32 products in any order inside one, n of them and a few
    more sums one after another, each rounded by up to a whole step."""
    return (40 + n) * 2 * U


def adapter_linear(x, ids, A, B, base, scale, one=1.0):
    """(out, v, bound of the kernel's error before the last rounding)"""
    x, A, B = x.double(), A.double(), B.double()
    n, R, K = A.shape
    M, N = x.shape[0], B.shape[1]
    out = torch.zeros(M, N, dtype=torch.float64, device=x.device) if base is None else base.double().clone()
    v = torch.zeros(M, R, dtype=torch.float64, device=x.device)
    bound = out.abs() * U
    for a in range(n):
        at = (ids == a).nonzero().flatten()
        if not at.numel():
            continue
        s = one if scale is None else float(scale[a])
        v[at] = x[at] @ A[a].t()
        out[at] += s * (v[at] @ B[a].t())
        dv = chain(K / 256) * (x[at].abs() @ A[a].abs().t()) + (2.0 ** -16 + 2 * U) * v[at].abs()
        bound[at] += abs(s) * ((dv + chain(R / 16) * v[at].abs()) @ B[a].abs().t()) + U * out[at].abs()
    return out, v, bound


def adapter_backward(x, ids, A, B, v, dy, base, scale):
    """(dx, dA, dB) and the bounds of the kernel's errors, dx's before its last rounding"""
    n, R, K = A.shape
    N = B.shape[1]
    dx, w, bound = adapter_linear(dy, ids, B.double().transpose(1, 2), A.double().transpose(1, 2), base, scale)
    dA, dB = torch.zeros_like(A, dtype=torch.float64), torch.zeros_like(B, dtype=torch.float64)
    bA, bB = torch.zeros_like(dA), torch.zeros_like(dB)
    x, dy, v = x.double(), dy.double(), v.double()
    for a in range(n):
        at = (ids == a).nonzero().flatten()
        if not at.numel():
            continue
        s = 1.0 if scale is None else float(scale[a])
        steps = chain(3 * at.numel() / 32 + 16) + 2 * U
        dA[a], dB[a] = s * (w[at].t() @ x[at]), s * (dy[at].t() @ v[at])
        dw = chain(N / 256) * (dy[at].abs() @ B[a].double().abs())
        bA[a] = abs(s) * ((dw + steps * w[at].abs()).t() @ x[at].abs())
        bB[a] = abs(s) * steps * (dy[at].abs().t() @ v[at].abs())
    return (dx, dA, dB), (bound, bA, bB)
