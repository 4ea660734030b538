"""The measured cases of six operators: expert selection from router logits and its gradient, MXFP4 quantization, the
dense and the grouped MXFP4 product, and gradient clipping by the global norm.

``run`` computes each in a plain form of elementary torch operations, or, where ``own`` is true, through
``nvfp4_moe_expert_sort_amd``.  ``exact`` gives the same values from the definitions in 64 bits."""
import math
import random

import torch

own = False

FLT_MAX = 3.4028234663852886e38
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEV = "cuda" if torch.cuda.is_available() else "cpu"


def listed():
    return [
        # one decode step of a few requests through this repository's router (128 experts, top 8): latency
        dict(name="select_decode", op="select", T=5, E=128, K=8, G=1, TG=1, top2=False, sigmoid=False, renorm=True,
             bias=False, scale=1.0, bf16=False),
        # a prefill batch through a router with sigmoid scores, a balance bias and groups of experts
        dict(name="select_prefill_grouped", op="select", T=16384, E=256, K=8, G=8, TG=4, top2=True, sigmoid=True,
             renorm=True, bias=True, scale=2.5, bf16=False),
        # a training batch's gradient with renormalised sigmoid weights: nonzero at the chosen experts only
        dict(name="select_backward_sparse", op="select_backward", T=4096, E=256, K=8, sigmoid=True, renorm=True,
             scale=2.5, bf16=False),
        # a large, ragged batch with weights of the softmax over all experts, logits and gradient in BF16
        dict(name="select_backward_dense", op="select_backward", T=32749, E=128, K=8, sigmoid=False, renorm=False,
             scale=1.0, bf16=True),
        # activations of one prefill batch, a row count that fills no tile, to MXFP4 and back
        dict(name="quantize_activations", op="quantize", rows=4099, cols=2048, up=False),
        # a quarter of the experts' first weights, block scales rounded up, to MXFP4 and back
        dict(name="quantize_weights", op="quantize", rows=49152, cols=2048, up=True),
        # one decode step of a few requests through a dense projection: reading the weights is the work
        dict(name="linear_decode", op="linear", M=7, N=4096, K=2048),
        # a training or prefill batch through a dense projection: the matrix cores are the work
        dict(name="linear_prefill", op="linear", M=8192, N=4096, K=4096),
        # 64 decode requests at top 8 over 128 experts of this repository's layer: a few rows an expert, some none
        dict(name="grouped_decode", op="grouped", R=512, E=128, N=1536, K=2048, skew=0.5),
        # 4096 tokens at top 8 over the same experts, uneven
        dict(name="grouped_prefill", op="grouped", R=32768, E=128, N=1536, K=2048, skew=0.3),
        # the small tensors of a model (norms, biases, routers) in both types, odd sizes
        dict(name="clip_many_small", op="clip", sizes=7, count=61, most=65537, bf16=True, max_norm=1.0),
        # the FP32 weight gradients of this repository's expert layer and its router
        dict(name="clip_expert_layer", op="clip", sizes=0, count=0, most=0, bf16=False, max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "select_backward", "quantize", "linear", "grouped", "clip"])
    if op == "select":
        T = _log(rng, 1, 16384)
        G = rng.choice([1, 1, 2, 4, 8])
        E = G * rng.randint(max(1, 8 // G), 256 // G)
        TG = rng.randint(1, G)
        bias, sigmoid = rng.random() < 0.6, rng.random() < 0.5
        return dict(op=op, T=T, E=E, K=rng.randint(1, min(8, TG * (E // G))), G=G, TG=TG, top2=rng.random() < 0.5,
                    sigmoid=sigmoid, renorm=rng.random() < 0.7, bias=bias, scale=rng.choice([1.0, 2.5]),
                    bf16=rng.random() < 0.4)
    if op == "select_backward":
        E = rng.randint(8, 256)
        return dict(op=op, T=_log(rng, 1, 4096 if E > 128 else 16384), E=E, K=rng.randint(2, 8),
                    sigmoid=rng.random() < 0.5, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    bf16=rng.random() < 0.5)
    if op == "quantize":
        cols = 32 * rng.randint(1, 256)
        return dict(op=op, rows=_log(rng, 1, (49152 * 2048) // cols // 4), cols=cols, up=rng.random() < 0.5)
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 6000), N=rng.randint(1, 4096), K=32 * rng.randint(1, 128))
    if op == "grouped":
        E = rng.choice([1, 3, 8, 60, 64, 128])
        return dict(op=op, R=_log(rng, 1, 8192), E=E, N=rng.randint(1, 1536), K=32 * rng.randint(1, 64),
                    skew=rng.choice([0.0, 0.3, 1.0]))
    return dict(op="clip", sizes=rng.randint(1, 1 << 20), count=_log(rng, 1, 60), most=_log(rng, 16, 1 << 20),
                bf16=rng.random() < 0.5, max_norm=rng.choice([0.1, 1.0, 1e6]))


def _grad_shapes(case):
    """[(shape, is BF16)] of a clip case: the expert layer's gradients, or `count` odd sizes up to `most`."""
    if not case["count"]:
        return [((128, 1536, 2048), False), ((128, 2048, 768), False), ((128, 2048), False)]
    r = random.Random(case["sizes"])
    return [((_log(r, 1, case["most"]),), case["bf16"] and r.random() < 0.5) for _ in range(case["count"])]


def work(case):
    op = case["op"]
    if op == "select":
        T, E, K = case["T"], case["E"], case["K"]
        return {"bytes": T * E * (2 if case["bf16"] else 4) + 8 * T * K + (4 * E if case["bias"] else 0),
                "flops": 4 * T * E}
    if op == "select_backward":
        T, E, K = case["T"], case["E"], case["K"]
        size = 2 if case["bf16"] else 4
        dense = not case["sigmoid"] and not case["renorm"]  # else the logits matter at the chosen experts only
        return {"bytes": T * E * size + T * (E if dense else K) * size + 8 * T * K, "flops": (6 * E if dense else 10 * K) * T}
    if op == "quantize":  # values read, codes and scales written; codes and scales read, values written
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * (2 * n + n // 2 + n // 32), "flops": 4 * n}
    if op in ("linear", "grouped"):
        M, N, K, E = case.get("M", case.get("R")), case["N"], case["K"], case.get("E", 1)
        used = min(E, M)  # an expert without rows needs none of its weights
        return {"bytes": used * N * K * 17 // 32 + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    n = sum(math.prod(s) * (2 if b else 4) for s, b in _grad_shapes(case))
    return {"bytes": 3 * n, "flops": 3 * sum(math.prod(s) for s, _ in _grad_shapes(case))}


def _normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * std


def _inputs(case, seed):
    """The tensors that a case computes on, from the seed alone."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    if op in ("select", "select_backward"):
        T, E, K = case["T"], case["E"], case["K"]
        logits = _normal((T, E), gen, 1.5)
        if case["bf16"]:
            logits = logits.to(torch.bfloat16)
        out = {"logits": logits}
        if op == "select":
            out["bias"] = _normal((E,), gen, 0.05) if case["bias"] else None
        else:
            ids = torch.sort(logits.double(), dim=1, descending=True, stable=True)[1][:, :K]
            out |= {"ids": ids.to(torch.int32).contiguous(), "dprobs": _normal((T, K), gen, 1e-2)}
        return out
    if op == "quantize":
        x = _normal((case["rows"], case["cols"]), gen)
        x *= torch.where(torch.rand((1, case["cols"]), generator=gen, device=DEV) < 0.01, 50.0, 1.0)  # outlier channels
        return {"x": x.to(torch.bfloat16)}
    if op in ("linear", "grouped"):
        M, N, K, E = case.get("M", case.get("R")), case["N"], case["K"], case.get("E", 1)
        x = _normal((M, K), gen)
        x *= torch.where(torch.rand((1, K), generator=gen, device=DEV) < 0.01, 20.0, 1.0)
        out = {"x": x.to(torch.bfloat16), "w": _normal((E, N, K), gen, 0.02).to(torch.bfloat16)}
        if op == "grouped":
            popularity = _normal((E,), gen, case["skew"] + 1e-6)
            expert = (popularity + -torch.log(-torch.log(torch.rand((M, E), generator=gen, device=DEV)))).argmax(1)
            out["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
            out["offsets"][1:] = torch.bincount(expert, minlength=E).cumsum(0)
        return out
    return {"grads": [_normal(s, gen, 1e-3 + 1e-2 * (i % 3)).to(torch.bfloat16 if b else torch.float32)
                      for i, (s, b) in enumerate(_grad_shapes(case))]}


# --- plain forms ------------------------------------------------------------------------------------

def _scores(logits, sigmoid):
    """(usable, clean logits with -inf where unusable, scores), in 64 bits: they are compared next to a border."""
    l = logits.double()
    usable = ~torch.isnan(l) & (l != -math.inf)
    l = torch.where(usable, l.clamp(max=FLT_MAX), -math.inf)
    if sigmoid:
        return usable, l, torch.where(usable, 1 / (1 + torch.exp(-l)), 0.0)
    top = l.max(1, keepdim=True)[0].clamp(min=-FLT_MAX)
    e = torch.exp(l - top)
    return usable, l, e / e.sum(1, keepdim=True).clamp(min=1e-300)


def _weights(l, s, live, sigmoid, renorm):
    """Weights of the chosen experts: l, s and live [T, K]."""
    if not renorm:
        return torch.where(live, s, 0.0)
    top = torch.where(live, l, -math.inf).max(1, keepdim=True)[0].clamp(min=-FLT_MAX)
    if sigmoid:  # sigma times e^-min(top, 0): the sum does not vanish
        shift = top.clamp(max=0)
        w = torch.where(l < 0, torch.exp(l.clamp(max=0) - shift) / (1 + torch.exp(l.clamp(max=0))), s)
    else:
        w = torch.exp(l - top)
    w = torch.where(live, w, 0.0)
    return w / w.sum(1, keepdim=True).clamp(min=1e-300)


def _plain_select(st):
    c, bias = st["case"], st["bias"]
    usable, l, s = _scores(st["logits"], c["sigmoid"])
    T, E, G = c["T"], c["E"], c["G"]
    b = torch.zeros(E, dtype=torch.float64, device=l.device) if bias is None else bias.double().clamp(max=FLT_MAX)
    live = usable & ~torch.isnan(b) & (b != -math.inf)
    v = torch.where(live, l if bias is None else s + b, -1e300)
    if G > 1:
        if c["top2"]:
            two = torch.where(live, s + b, -math.inf).view(T, G, E // G).sort(dim=2, descending=True)[0][:, :, :2]
            group = torch.where(two[..., :1] == -math.inf, -math.inf, torch.where(two == -math.inf, 0.0, two)).sum(2)
        else:
            group = torch.where(live, v, -math.inf).view(T, G, E // G).max(2)[0]
        kept = group.sort(dim=1, descending=True, stable=True)[1][:, :c["TG"]]
        mask = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        v = torch.where(mask.repeat_interleave(E // G, 1), v, -math.inf)
    ids = v.sort(dim=1, descending=True, stable=True)[1][:, :c["K"]]
    take = lambda t: t.gather(1, ids)  # noqa: E731
    w = _weights(take(l), take(s), take(live), c["sigmoid"], c["renorm"])
    return {"ids": ids.to(torch.int32), "probs": (w * c["scale"]).float()}


def _plain_select_backward(st):
    c, ids, dp = st["case"], st["ids"].long(), st["dprobs"].double()
    usable, l, s = _scores(st["logits"], c["sigmoid"])
    lk, sk, live = l.gather(1, ids), s.gather(1, ids), usable.gather(1, ids)
    w = _weights(lk, sk, live, c["sigmoid"], c["renorm"])
    mean = (w * dp).sum(1, keepdim=True)
    if c["renorm"]:
        d = w * (dp - mean) * ((1 - sk) if c["sigmoid"] else 1.0)
    elif c["sigmoid"]:
        d = w * dp * (1 - sk)
    else:
        d = w * dp
    out = torch.zeros_like(l).scatter_add_(1, ids, d * c["scale"])
    if not c["renorm"] and not c["sigmoid"]:
        out = out - c["scale"] * s * mean
    return {"dlogits": out.to(st["logits"].dtype)}


def _plain_mxfp4(x, up):
    """The values that x [..., C] has in MXFP4, in 32 bits."""
    b = x.float().unflatten(-1, (-1, 32))
    a = b.abs()
    mant, e = torch.frexp(a.amax(-1, keepdim=True))  # amax = mant 2^e, mant in [1/2, 1)
    k = (e - 3 + ((mant > 0.75).int() if up else 0)).clamp(min=-127)
    unit = torch.exp2(k.double())
    q = a * torch.exp2(-k.double()).float()
    code = ((q > 0.25).int() + (q >= 0.75).int() + (q > 1.25).int() + (q >= 1.75).int() + (q > 2.5).int()
            + (q >= 3.5).int() + (q > 5.0).int())
    value = torch.tensor(E2M1, device=x.device)[code] * unit.float()
    return torch.where(b < 0, -value, value).flatten(-2)


def _plain_grouped(st):
    x, off, E = _plain_mxfp4(st["x"], False), st["offsets"].long(), st["case"]["E"]
    row = torch.arange(x.shape[0], device=x.device)
    e = torch.searchsorted(off[1:], row, right=True)
    slot = row - off[e]
    chunks = torch.zeros(E, st["most"], x.shape[1], device=x.device)
    chunks[e, slot] = x
    return torch.bmm(chunks, st["wt"])[e, slot].to(torch.bfloat16)


def _plain_clip(st):
    norm = torch.stack([g.double().square().sum() for g in st["grads"]]).sum().sqrt()
    coef = torch.where(norm > st["case"]["max_norm"], st["case"]["max_norm"] / norm, 1.0)
    coef = torch.where(torch.isfinite(norm), coef, 1.0).float()
    return {"norm": norm.view(1), "grads": [(g.float() * coef).to(g.dtype) for g in st["grads"]]}


# --- the measured calls -----------------------------------------------------------------------------

def prepare(case, seed):
    st = {"case": case} | _inputs(case, seed)
    op = case["op"]
    if op in ("linear", "grouped"):
        # a program keeps its weights quantized: the library's handle, or their values, laid out for the plain product
        w = st.pop("w")
        if own:
            import nvfp4_moe_expert_sort_amd as m
            st["wq"] = m.Mxfp4Weights(*w.shape, device=w.device).quantize_from(w)
            st["ws"] = m.mxfp4_alloc_workspace(*st["x"].shape, n_mats=w.shape[0], device=w.device)
        else:
            st["wt"] = _plain_mxfp4(w, False).transpose(1, 2).contiguous()
            if op == "grouped":
                st["most"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())
    if op == "clip" and own:
        import nvfp4_moe_expert_sort_amd as m
        st["clipped"] = [torch.empty_like(g) for g in st["grads"]]
        st["set"] = m.GradSet(st["grads"], st["clipped"])
    return st


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import nvfp4_moe_expert_sort_amd as m
        if op == "select":
            ids, probs = m.router_select(
                state["logits"], case["K"], bias=state["bias"], score=m.SCORE_SIGMOID if case["sigmoid"] else m.SCORE_SOFTMAX,
                renormalize=case["renorm"], scale=case["scale"], n_groups=case["G"], top_groups=case["TG"],
                group_score=m.GROUP_TOP2 if case["top2"] else m.GROUP_MAX)
            return {"ids": ids, "probs": probs}
        if op == "select_backward":
            return {"dlogits": m.router_select_backward(
                state["logits"], state["ids"], state["dprobs"], score=m.SCORE_SIGMOID if case["sigmoid"] else m.SCORE_SOFTMAX,
                renormalize=case["renorm"], scale=case["scale"])}
        if op == "quantize":
            codes, scales = m.mxfp4_quantize(state["x"], scale_round=m.MXFP4_SCALE_RU if case["up"] else m.MXFP4_SCALE_FLOOR)
            return {"values": m.mxfp4_dequantize(codes, scales)}
        if op == "linear":
            return {"out": m.mxfp4_linear(state["x"], state["wq"], workspace=state["ws"])}
        if op == "grouped":
            return {"out": m.mxfp4_grouped_linear(state["x"], state["offsets"], state["wq"], workspace=state["ws"])}
        return {"norm": m.clip_grad_norm(state["set"], case["max_norm"]), "grads": state["clipped"]}
    if op == "select":
        return _plain_select(state)
    if op == "select_backward":
        return _plain_select_backward(state)
    if op == "quantize":
        return {"values": _plain_mxfp4(state["x"], case["up"]).to(torch.bfloat16)}
    if op == "linear":
        return {"out": torch.matmul(_plain_mxfp4(state["x"], False), state["wt"][0]).to(torch.bfloat16)}
    if op == "grouped":
        return {"out": _plain_grouped(state)}
    return _plain_clip(state)


# --- the definitions in 64 bits ----------------------------------------------------------------------

def _nearest_mxfp4(x, up):
    """x [..., C] in MXFP4, in 64 bits: the scale found among the powers of two, each element by its distances."""
    x = x.double().unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1, keepdim=True)
    k = torch.floor(torch.log2(amax.clamp(min=2.0 ** -140)))
    k = k - (torch.exp2(k) > amax).double() + (torch.exp2(k + 1) <= amax).double() - 2
    if up:
        k = k + (6 * torch.exp2(k) < amax).double()
    unit = torch.exp2(k.clamp(min=-127))
    best, far = torch.zeros_like(x), torch.full_like(x, math.inf)
    for code, v in enumerate(E2M1):
        d = (x.abs() / unit - v).abs()
        better = (d < far) | ((d == far) & (code % 2 == 0))  # ties to the even code
        best, far = torch.where(better, v, best), torch.where(better, d, far)
    return (torch.sign(x) * best * unit).flatten(-2)


def _exact_selected(case, l, s, b, live):
    """The chosen ids [T, K] by counting, for each expert, those that come before it."""
    T, E, G, K = case["T"], case["E"], case["G"], case["K"]
    v = l if b is None else s + b
    w = torch.where(live, s if b is None else s + b, -math.inf)
    kept = torch.ones(T, E, dtype=torch.bool, device=l.device)
    if G > 1:
        n = E // G
        if case["top2"]:
            first, at = w.view(T, G, n).max(2)
            rest = w.view(T, G, n).clone().scatter_(2, at[..., None], -math.inf)
            second = rest.max(2)[0]
            group = first + torch.where(second == -math.inf, 0.0, second)
        else:
            group = torch.where(live, v, -math.inf).view(T, G, n).max(2)[0]
        g = torch.arange(G, device=l.device)
        before = (group[:, None, :] > group[:, :, None]) | ((group[:, None, :] == group[:, :, None]) & (g[None, :] < g[:, None]))
        kept = (before.sum(2) < case["TG"])[:, :, None].expand(T, G, n).reshape(T, E)
    e = torch.arange(E, device=l.device)
    ids = torch.empty(T, K, dtype=torch.int64, device=l.device)
    for t0 in range(0, T, 2048):
        t = slice(t0, t0 + 2048)
        a, va, ka = live[t], torch.where(live[t], v[t], 0.0), kept[t]
        less = (va[:, None, :] > va[:, :, None]) | ((va[:, None, :] == va[:, :, None]) & (e[None, :] < e[:, None]))
        less = torch.where(a[:, None, :] == a[:, :, None], less, a[:, None, :] & ~a[:, :, None])
        rank = torch.where(ka, (less & ka[:, None, :]).sum(2), E)
        ids[t] = rank.sort(dim=1, stable=True)[1][:, :K]
    return ids


def exact(case, seed):
    st, op = _inputs(case, seed), case["op"]
    if op in ("select", "select_backward"):
        l = st["logits"].double()  # the inputs are finite
        one = torch.ones_like(l, dtype=torch.bool)
        s = torch.special.expit(l) if case["sigmoid"] else torch.softmax(l, 1)
        ids = st["ids"].long() if op == "select_backward" else _exact_selected(
            case, l, s, None if st["bias"] is None else st["bias"].double(), one)
        p = s.gather(1, ids)
        total = p.sum(1, keepdim=True) if case["renorm"] else 1.0
        if op == "select":
            return {"ids": ids.to(torch.int32), "probs": case["scale"] * p / total}
        dp = st["dprobs"].double() * case["scale"]
        dk = (dp - (dp * p / total).sum(1, keepdim=True)) / total if case["renorm"] else dp
        ds = torch.zeros_like(s).scatter_add_(1, ids, dk)
        return {"dlogits": ds * s * (1 - s) if case["sigmoid"] else s * (ds - (ds * s).sum(1, keepdim=True))}
    if op == "quantize":
        return {"values": torch.cat([_nearest_mxfp4(part, case["up"]) for part in st["x"].split(8192)])}
    if op == "linear":
        return {"out": _nearest_mxfp4(st["x"], False) @ _nearest_mxfp4(st["w"][0], False).t().contiguous()}
    if op == "grouped":
        x, off = _nearest_mxfp4(st["x"], False), st["offsets"].tolist()
        return {"out": torch.cat([x[a:b] @ _nearest_mxfp4(w, False).t().contiguous()
                                  for a, b, w in zip(off, off[1:], st["w"])])}
    squares = [(g.double() ** 2).sum().item() for g in st["grads"]]
    norm = math.sqrt(math.fsum(squares))
    coef = case["max_norm"] / norm if norm > case["max_norm"] else 1.0
    return {"norm": torch.tensor([norm], dtype=torch.float64, device=DEV), "grads": [g.double() * coef for g in st["grads"]]}
