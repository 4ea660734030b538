"""The measured cases of four operators: the router's balance loss with its per-expert counts, its gradient, low-rank
adapters of many requests beside a shared projection, and their gradients.

``run`` computes each in a plain form of elementary torch operations, or, where ``own`` is true, through
``nvfp4_moe_expert_sort_amd``.  ``exact`` gives the same values from the definitions in 64 bits."""
import math

import torch

own = False

COEF = 0.01  # of the balance loss
DEV = "cuda" if torch.cuda.is_available() else "cpu"


def listed():
    return [
        # a small fine-tuning batch through this repository's router (128 experts, top 8): latency
        dict(name="balance_small", op="balance", T=61, E=128, K=8, S=1, sigmoid=False, bf16=False),
        # a packed pretraining batch of ragged sequences, each balanced by itself, sigmoid scores of 256 experts
        dict(name="balance_packed", op="balance", T=16384, E=256, K=8, S=13, sigmoid=True, bf16=False),
        # a training batch's gradient, added to the one that the weights of the chosen experts give
        dict(name="balance_backward", op="balance_backward", T=4096, E=128, K=8, S=1, sigmoid=False, bf16=False, add=True),
        # a large, ragged batch of packed sequences, logits and gradient in BF16
        dict(name="balance_backward_packed", op="balance_backward", T=32749, E=128, K=8, S=40, sigmoid=True, bf16=True,
             add=False),
        # one decode step of a few requests, each with an adapter of its own: latency
        dict(name="adapter_decode", op="adapter", M=5, K=2048, N=4096, R=16, n=8, rows="each", none=0.0),
        # one decode step of many requests over many adapters, some without one
        dict(name="adapter_decode_many", op="adapter", M=200, K=4096, N=4096, R=32, n=64, rows="each", none=0.1),
        # prefill of a few long requests through a dense projection
        dict(name="adapter_prefill", op="adapter", M=8192, K=4096, N=4096, R=16, n=8, rows="requests", none=0.0),
        # a ragged prefill batch, a high rank, requests without an adapter between the others
        dict(name="adapter_prefill_rank64", op="adapter", M=4099, K=2048, N=4096, R=64, n=5, rows="requests", none=0.2),
        # adapters of this repository's 128 experts beside their first product: 4096 tokens at top 8, sorted by expert
        dict(name="adapter_experts", op="adapter", M=32768, K=2048, N=1536, R=16, n=128, rows="experts", none=0.0),
        # a fine-tuning step of one adapter on a small batch
        dict(name="adapter_backward_one", op="adapter_backward", M=1021, K=2048, N=4096, R=16, n=1, rows="requests",
             none=0.0),
        # a step that trains a few adapters of a high rank at once
        dict(name="adapter_backward_rank64", op="adapter_backward", M=8192, K=4096, N=4096, R=64, n=4, rows="requests",
             none=0.0),
        # the gradients of the experts' adapters
        dict(name="adapter_backward_experts", op="adapter_backward", M=32768, K=2048, N=1536, R=16, n=128,
             rows="experts", none=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "balance_backward", "adapter", "adapter_backward"])
    if op in ("balance", "balance_backward"):
        E, T = rng.randint(4, 256), _log(rng, 1, 16384)
        case = dict(op=op, T=T, E=E, K=rng.randint(1, min(8, E)), S=rng.choice([1, 1, _log(rng, 1, min(T, 64))]),
                    sigmoid=rng.random() < 0.5, bf16=rng.random() < 0.4)
        return case | ({"add": rng.random() < 0.5} if op == "balance_backward" else {})
    return dict(op=op, M=_log(rng, 1, 6000), K=8 * rng.randint(4, 512), N=8 * rng.randint(4, 512), R=8 * rng.randint(1, 8),
                n=rng.choice([1, 2, 7, 32, 100]), rows=rng.choice(["each", "requests", "experts"]),
                none=rng.choice([0.0, 0.0, 0.3]))


def work(case):
    if case["op"] in ("balance", "balance_backward"):
        T, E, K, S = case["T"], case["E"], case["K"], case["S"]
        size = 2 if case["bf16"] else 4
        if case["op"] == "balance":
            return {"bytes": T * E * size + 4 * T * K + 4 * S * E, "flops": 6 * T * E}
        return {"bytes": T * E * size * (3 if case["add"] else 2) + 4 * S * E, "flops": 8 * T * E}
    M, K, N, R, n = (case[x] for x in ("M", "K", "N", "R", "n"))
    used = min(n, M)  # an adapter without rows need not be read
    if case["op"] == "adapter":
        return {"bytes": 2 * M * (K + 2 * N) + 4 * M + 2 * used * R * (K + N), "flops": 2 * M * R * (K + N)}
    return {"bytes": 2 * M * (3 * K + N) + 4 * M * (R + 1) + 2 * used * R * (K + N) + 4 * n * R * (K + N),
            "flops": 4 * M * R * (K + N)}


def _normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * std


def _cuts(rows, parts, gen):
    """Offsets [parts + 1] of consecutive parts of random lengths that hold all rows."""
    cut = torch.rand(parts - 1, generator=gen, device=DEV).mul(rows + 1).long().clamp(max=rows).sort()[0]
    ends = torch.tensor([0, rows], device=DEV)
    return torch.cat([ends[:1], cut, ends[1:]])


def _adapter_ids(case, gen):
    """The adapter of each row, -1 for none."""
    M, n = case["M"], case["n"]
    if case["rows"] == "experts":  # sorted, of uneven popularity
        popularity = _normal((n,), gen, 0.3)
        noise = -torch.log(-torch.log(torch.rand((M, n), generator=gen, device=DEV)))
        ids = (popularity + noise).argmax(1).sort()[0]
    else:
        parts = M if case["rows"] == "each" else min(M, 2 * n + 1)
        ids = torch.randint(0, n, (parts,), generator=gen, device=DEV)
        if case["none"]:
            ids = torch.where(torch.rand(parts, generator=gen, device=DEV) < case["none"], -1, ids)
        if case["rows"] == "requests":
            ids = ids[torch.searchsorted(_cuts(M, parts, gen)[1:-1], torch.arange(M, device=DEV), right=True)]
    return ids.to(torch.int32).contiguous()


def _inputs(case, seed):
    """The tensors that a case computes on, from the seed alone."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] in ("balance", "balance_backward"):
        T, E, K, S = case["T"], case["E"], case["K"], case["S"]
        kind = torch.bfloat16 if case["bf16"] else torch.float32
        out = {"logits": (_normal((T, E), gen, 1.5) + _normal((1, E), gen, 0.5)).to(kind)}  # some experts are preferred
        out["ids"] = torch.sort(out["logits"].double(), dim=1, descending=True, stable=True)[1][:, :K].to(torch.int32).contiguous()
        out["offsets"] = _cuts(T, S, gen).to(torch.int32) if S > 1 else None
        if case["op"] == "balance_backward":
            out["dloss"] = 0.5 + torch.rand(1, generator=gen, device=DEV)
            out["counts"] = _counts(out["ids"], out["offsets"], E)
            out["add"] = _normal((T, E), gen, COEF / (T * E)).to(kind) if case["add"] else None
        return out
    M, K, N, R, n = (case[x] for x in ("M", "K", "N", "R", "n"))
    bf16 = torch.bfloat16
    out = {"x": _normal((M, K), gen).to(bf16), "ids": _adapter_ids(case, gen),
           "A": _normal((n, R, K), gen, K ** -0.5).to(bf16), "B": _normal((n, N, R), gen, 0.1).to(bf16),
           "scale": 0.5 + 1.5 * torch.rand(n, generator=gen, device=DEV)}
    if case["op"] == "adapter":
        out["base"] = _normal((M, N), gen).to(bf16)  # what the shared projection gave
    else:
        out["dy"] = _normal((M, N), gen, 1e-2).to(bf16)
        out["base"] = _normal((M, K), gen, 1e-2).to(bf16)  # the gradient through the shared projection
        every = (out["x"].float() @ out["A"].float().view(n * R, K).t().contiguous()).view(M, n, R)
        v = every[torch.arange(M, device=DEV), out["ids"].long().clamp(min=0)]
        out["v"] = torch.where(out["ids"][:, None] >= 0, v, 0.0)  # the forward's
    return out


# --- plain forms ------------------------------------------------------------------------------------


def _sequences(T, offsets):
    """(first row of each sequence and the end, the sequence of each row)"""
    if offsets is None:
        return torch.tensor([0, T], device=DEV), torch.zeros(T, dtype=torch.int64, device=DEV)
    return offsets.long(), torch.searchsorted(offsets[1:].long(), torch.arange(T, device=DEV), right=True)


def _counts(ids, offsets, E):
    T, K = ids.shape
    off, seq = _sequences(T, offsets)
    S = off.numel() - 1
    at = (seq[:, None] * E + ids.long()).flatten()
    return torch.zeros(S * E, dtype=torch.int32, device=DEV).index_add_(0, at, torch.ones_like(at, dtype=torch.int32)).view(S, E)


def _probabilities(logits, sigmoid):
    """(p, sigma or None): the softmax, or sigmoids divided by their sum."""
    l = logits.float()
    if sigmoid:
        s = 1 / (1 + torch.exp(-l))
        return s / s.sum(1, keepdim=True), s
    e = torch.exp(l - l.max(1, keepdim=True)[0])
    return e / e.sum(1, keepdim=True), None


def _plain_balance(st):
    c, logits = st["case"], st["logits"]
    T, E = logits.shape
    off, seq = _sequences(T, st["offsets"])
    counts = _counts(st["ids"], st["offsets"], E)
    f = counts.float() * (E / c["K"]) / (off[1:] - off[:-1]).clamp(min=1)[:, None]
    p = _probabilities(logits, c["sigmoid"])[0]
    return {"loss": ((f[seq] * p).double().sum() * (COEF / T)).float().view(1), "counts": counts}


def _plain_balance_backward(st):
    c, logits = st["case"], st["logits"]
    T, E = logits.shape
    off, seq = _sequences(T, st["offsets"])
    f = (st["counts"].float() * (E / c["K"]) / (off[1:] - off[:-1]).clamp(min=1)[:, None])[seq]
    p, s = _probabilities(logits, c["sigmoid"])
    d = p * (f - (f * p).sum(1, keepdim=True)) * (st["dloss"] * (COEF / T))
    if s is not None:
        d = d * (1 - s)
    if st["add"] is not None:
        d = d + st["add"].float()
    return {"dlogits": d.to(logits.dtype)}


def _chunks(st, rows):
    """rows [M, C] in 32 bits, those of each adapter in a chunk of its own: [n, most, C]."""
    n, (live, a, slot) = st["case"]["n"], st["at"]
    out = torch.zeros(n, st["most"], rows.shape[1], device=DEV)
    out[a, slot] = rows[live].float()
    return out


def _back(st, base, chunks):
    """base in 32 bits, with each adapter's chunk added to its rows, in BF16."""
    live, a, slot = st["at"]
    out = base.float()
    out[live] += chunks[a, slot]
    return out.to(torch.bfloat16)


def _place(st):
    """The rows with an adapter, each one's adapter, and its place among that adapter's."""
    live = st["ids"].long().sort(stable=True)[1][st["case"]["M"] - st["live"]:]  # (those without one come first)
    a = st["ids"].long()[live]
    first = torch.searchsorted(a, torch.arange(st["case"]["n"], device=DEV))
    return live, a, torch.arange(st["live"], device=DEV) - first[a]


def _plain_adapter(st):
    st = st | {"at": _place(st)}
    v = torch.bmm(_chunks(st, st["x"]), st["At"]) * st["scale"][:, None, None]
    return {"out": _back(st, st["base"], torch.bmm(v, st["Bt"]))}


def _plain_adapter_backward(st):
    st = st | {"at": _place(st)}
    x, dy, v, scale = _chunks(st, st["x"]), _chunks(st, st["dy"]), _chunks(st, st["v"]), st["scale"][:, None, None]
    w = torch.bmm(dy, st["B"].float()) * scale
    dx = _back(st, st["base"], torch.bmm(w, st["A"].float()))
    dA = torch.bmm(w.transpose(1, 2).contiguous(), x)
    dB = torch.bmm(dy.transpose(1, 2).contiguous(), v) * scale
    return {"dx": dx, "dA": dA, "dB": dB}


# --- the measured calls -----------------------------------------------------------------------------

def prepare(case, seed):
    st = {"case": case} | _inputs(case, seed)
    if case["op"] in ("adapter", "adapter_backward"):
        if own:
            import nvfp4_moe_expert_sort_amd as m
            st["ws"] = m.adapter_alloc_workspace(case["M"], case["K"], case["N"], case["R"], case["n"],
                                                 backward=case["op"] == "adapter_backward")
        else:  # sizes of the chunks, and for the forward pass the weights laid out for the plain products
            count = torch.bincount(st["ids"][st["ids"] >= 0].long(), minlength=case["n"])
            st["live"], st["most"] = int(count.sum()), max(1, int(count.max()))
            if case["op"] == "adapter":
                st["At"], st["Bt"] = (st[k].float().transpose(1, 2).contiguous() for k in ("A", "B"))
    return st


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import nvfp4_moe_expert_sort_amd as m
        if op == "balance":
            loss, counts = m.router_balance_loss(
                state["logits"], state["ids"], COEF, score=m.SCORE_SIGMOID if case["sigmoid"] else m.SCORE_SOFTMAX,
                offsets=state["offsets"])
            return {"loss": loss, "counts": counts}
        if op == "balance_backward":
            return {"dlogits": m.router_balance_backward(
                state["logits"], state["counts"], case["K"], COEF, dloss=state["dloss"], add=state["add"],
                score=m.SCORE_SIGMOID if case["sigmoid"] else m.SCORE_SOFTMAX, offsets=state["offsets"])}
        if op == "adapter":
            return {"out": m.adapter_linear(state["x"], state["ids"], state["A"], state["B"], base=state["base"],
                                            scale=state["scale"], workspace=state["ws"])}
        dx, dA, dB = m.adapter_backward(state["x"], state["ids"], state["A"], state["B"], state["v"], state["dy"],
                                        base=state["base"], scale=state["scale"], workspace=state["ws"])
        return {"dx": dx, "dA": dA, "dB": dB}
    return {"balance": _plain_balance, "balance_backward": _plain_balance_backward, "adapter": _plain_adapter,
            "adapter_backward": _plain_adapter_backward}[op](state)


# --- the definitions in 64 bits ----------------------------------------------------------------------

def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] in ("balance", "balance_backward"):
        l = st["logits"].double()  # the inputs are finite
        T, E = l.shape
        ends = [0, T] if st["offsets"] is None else st["offsets"].tolist()
        s = torch.special.expit(l)
        p = s / s.sum(1, keepdim=True) if case["sigmoid"] else torch.softmax(l, 1)
        if case["op"] == "balance":
            counts, loss = torch.zeros(case["S"], E, dtype=torch.int32, device=DEV), 0.0
            for i, (a, b) in enumerate(zip(ends, ends[1:])):
                counts[i] = torch.bincount(st["ids"][a:b].flatten().long(), minlength=E).to(torch.int32)
                if b > a:
                    loss += float(counts[i].double() @ p[a:b].sum(0)) * E / (case["K"] * (b - a))
            return {"loss": torch.tensor([loss * COEF / T], dtype=torch.float64, device=DEV), "counts": counts}
        d = torch.zeros_like(l)
        for i, (a, b) in enumerate(zip(ends, ends[1:])):
            if b > a:
                f = st["counts"][i].double() * E / (case["K"] * (b - a))
                g = f - p[a:b] @ f[:, None]
                d[a:b] = p[a:b] * g * (1 - s[a:b] if case["sigmoid"] else 1.0)
        d = d * (st["dloss"].double() * COEF / T)
        return {"dlogits": d if st["add"] is None else d + st["add"].double()}
    A, B, x, scale = st["A"].double(), st["B"].double(), st["x"].double(), st["scale"].double()
    out = st["base"].double()
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for a in range(case["n"]):
        at = (st["ids"] == a).nonzero().flatten()
        if case["op"] == "adapter":
            out[at] += scale[a] * ((x[at] @ A[a].t().contiguous()) @ B[a].t().contiguous())
        else:
            dy = st["dy"][at].double()
            w = scale[a] * (dy @ B[a])
            out[at] += w @ A[a]
            dA[a] = w.t().contiguous() @ x[at]
            dB[a] = scale[a] * (dy.t().contiguous() @ st["v"][at].double())
    return {"out": out} if case["op"] == "adapter" else {"dx": out, "dA": dA, "dB": dB}
