"""The layer's neighbouring operators as measured cases: what a decoder runs
around the routed experts.

linear   y = act(x W^T + bias) [* (x Wu^T + bias_u)] + residual
         dense products next to the expert layer: the output projection that
         writes the residual stream, router logits, a shared or dense FFN of
         any width (gated), with the epilogue in the product.
route    expert choice from router logits: softmax or sigmoid scores, a
         selection bias, groups of experts, top-k, renormalised and scaled
         weights.

`own` False: the plain form in torch, fp32 (fp64 where choices are compared),
rounded once.  `own` True: the library's calls.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _lin(name, t, k, n, dtype="bf16", out="bf16", act="none", gated=False, bias=False, residual=False, pad=0):
    """pad: x is the first k columns of rows of k + pad (a slice of a wider projection)."""
    return dict(name=name, op="linear", t=t, k=k, n=n, dtype=dtype, out=out, act=act, gated=gated, bias=bias,
                residual=residual, pad=pad)


def _rt(name, t, e, top, score="softmax", dtype="f32", bias=False, groups=1, keep=1, group_score="max", renorm=True,
        scale=1.0, off=0):
    """off: experts out of service (selection bias -inf)."""
    return dict(name=name, op="route", t=t, e=e, top=top, score=score, dtype=dtype, bias=bias, groups=groups,
                keep=keep, group_score=group_score, renorm=renorm, scale=scale, off=off)


def listed():
    return [
        # one decoded token: the projection back into the residual stream
        _lin("proj_1_token", 1, 4096, 4096, residual=True),
        # one decoded token: router logits, the smallest product
        _lin("logits_1_token", 1, 4096, 512, out="f32", bias=True),
        # a few sequences decoded together, odd widths, a slice of a wider buffer
        _lin("odd_13_tokens", 13, 2040, 1001, dtype="f16", out="f16", act="gelu", bias=True, pad=72),
        # a decode batch through a gated FFN's first product
        _lin("gated_64_tokens", 64, 4096, 1024, act="silu", gated=True),
        # a short prompt through the FFN's second product, ragged
        _lin("down_250_tokens", 250, 1024, 4096, residual=True),
        # prompts: gated product of a wide dense FFN
        _lin("gated_2048_tokens", 2048, 4096, 4096, act="silu", gated=True),
        # a long prompt batch: bias and activation, the largest product
        _lin("wide_8192_tokens", 8192, 4096, 8192, act="gelu_tanh", bias=True),
        # one decoded token: 4 of 512 experts by softmax
        _rt("route_1_token", 1, 512, 4),
        # a decode batch: sigmoid scores, balance bias, groups
        _rt("route_groups_96_tokens", 96, 512, 8, score="sigmoid", bias=True, groups=16, keep=4, group_score="top2",
            scale=1.5),
        # prompts: the same choice for many tokens, some experts out of service
        _rt("route_groups_4096_tokens", 4096, 512, 8, score="sigmoid", bias=True, groups=16, keep=4,
            group_score="top2", scale=1.5, off=5),
        # a long prompt batch: softmax over all experts, raw weights, logits in 16 bits
        _rt("route_16384_tokens", 16384, 512, 10, dtype="bf16", renorm=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.6:
        while True:
            t, k, n = _log(rng, 1, 16384), 8 * _log(rng, 8, 2048), _log(rng, 16, 16384)
            step = rng.choice([1, 8, 64, 64])
            n = max(step, n // step * step)
            gated = rng.random() < 0.35
            if t * k * n * (2 if gated else 1) <= 8192 * 4096 * 8192:
                break
        dtype = rng.choice(["bf16", "bf16", "f16"])
        act = rng.choice(["silu", "gelu_tanh", "gelu"] if gated else ["none", "none", "silu", "gelu", "gelu_tanh", "relu"])
        c = _lin("", t, k, n, dtype, rng.choice([dtype, dtype, "f32"]), act, gated, rng.random() < 0.5,
                 rng.random() < 0.5, rng.choice([0, 0, 8 * rng.randint(1, 64)]))
    else:
        groups = rng.choice([1, 1, 4, 8, 16])
        e = groups * rng.choice([4, 12, 16, 24, 32]) if groups > 1 else rng.randint(8, 1024)
        keep = rng.randint(max(1, groups // 4), max(1, groups // 2))
        top = rng.randint(1, min(16, e // groups * keep))
        bias = rng.random() < 0.6
        c = _rt("", _log(rng, 1, 16384), e, top, rng.choice(["softmax", "sigmoid"]), rng.choice(["f32", "f32", "bf16"]),
                bias, groups, keep, rng.choice(["max", "top2"]), rng.random() < 0.7, rng.choice([1.0, 1.5, 2.5]),
                rng.randint(0, e // 8) if bias else 0)
    del c["name"]
    return c


def _inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": c}
    if c["op"] == "linear":
        dt = _DT[c["dtype"]]
        s["x"] = normal(c["t"], c["k"] + c["pad"], dtype=dt)[:, :c["k"]]
        s["w"] = normal(c["n"], c["k"], std=0.02, dtype=dt)
        s["wu"] = normal(c["n"], c["k"], std=0.02, dtype=dt) if c["gated"] else None
        s["bias"] = normal(c["n"], std=0.1) if c["bias"] else None
        s["bias_u"] = normal(c["n"], std=0.1) if c["bias"] and c["gated"] else None
        s["residual"] = normal(c["t"], c["n"], dtype=_DT[c["out"]]) if c["residual"] else None
    else:
        s["logits"] = normal(c["t"], c["e"], std=1.3, dtype=_DT[c["dtype"]])
        s["bias"] = None
        if c["bias"]:
            s["bias"] = normal(c["e"], std=0.05)
            s["bias"][torch.randperm(c["e"], generator=g, device="cuda")[:c["off"]]] = -math.inf
    return s


def prepare(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "linear":
        s["out"] = torch.empty(c["t"], c["n"], dtype=_DT[c["out"]], device="cuda")
    else:
        s["idx"] = torch.empty(c["t"], c["top"], dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(c["t"], c["top"], dtype=torch.float32, device="cuda")
    if own:
        import quantized_expert_ffn_03_b200 as M
        s["M"] = M
        if c["op"] == "linear":
            dtypes = {"bf16": M.MOE_BF16, "f16": M.MOE_F16, "f32": M.MOE_F32}
            acts = {"none": M.MOE_ACT_NONE, "silu": M.MOE_ACT_SILU, "gelu": M.MOE_ACT_GELU,
                    "gelu_tanh": M.MOE_ACT_GELU_TANH, "relu": M.MOE_ACT_RELU}
            s["cfg"] = M.linear_config(c["k"], c["n"], act=acts[c["act"]], gated=c["gated"], dtype=dtypes[c["dtype"]],
                                       out_dtype=dtypes[c["out"]])
            s["wts"] = M.linear_weights(s["cfg"], s["w"], bias=s["bias"], w_up=s["wu"], bias_up=s["bias_u"])
        else:
            s["cfg"] = M.route_config(
                c["e"], c["top"], score=M.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else M.MOE_SCORE_SOFTMAX,
                n_groups=c["groups"], topk_groups=c["keep"],
                group_score=M.MOE_GROUP_TOP2 if c["group_score"] == "top2" else M.MOE_GROUP_MAX,
                renormalise=c["renorm"], scale=c["scale"])
    return s


def _act(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v.clamp(min=0) if act == "relu" else v


def _linear_plain(s):
    x = s["x"].float()
    v = x @ s["w"].float().T
    if s["bias"] is not None:
        v = v + s["bias"]
    v = _act(v, s["case"]["act"])
    if s["wu"] is not None:
        u = x @ s["wu"].float().T
        v = v * (u if s["bias_u"] is None else u + s["bias_u"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(s["out"].dtype)


def _route_plain(s):
    """Choices are compared in fp64: the order of two scores a rounding apart is part of the result."""
    c = s["case"]
    t, e, g = c["t"], c["e"], c["groups"]
    v = s["logits"].double()
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-v))
    else:
        score = torch.exp(v - v.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    value = score if s["bias"] is None else score + s["bias"].double()
    inside = torch.ones(t, e, dtype=torch.bool, device=v.device)
    if g > 1:
        best = value.view(t, g, e // g).sort(dim=2, descending=True)[0]
        of_group = best[:, :, :2].sum(2) if c["group_score"] == "top2" else best[:, :, 0]
        kept = of_group.sort(dim=1, descending=True, stable=True)[1][:, :c["keep"]]
        inside = torch.zeros(t, g, dtype=torch.bool, device=v.device).scatter(1, kept, True)
        inside = inside.repeat_interleave(e // g, 1)
    order = value.sort(dim=1, descending=True, stable=True)[1]
    first = inside.gather(1, order).to(torch.int8).sort(dim=1, descending=True, stable=True)[1]
    idx = order.gather(1, first[:, :c["top"]])
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.to(torch.int32), (w * c["scale"]).float()


def run(s):
    if s["case"]["op"] == "linear":
        if own:
            s["M"].moe_linear_forward(s["cfg"], s["wts"], s["x"], s["out"], residual=s["residual"])
            return s["out"]
        return _linear_plain(s)
    if own:
        s["M"].moe_route_from_logits(s["cfg"], s["logits"], s["idx"], s["weights"], select_bias=s["bias"])
        return s["idx"], s["weights"]
    return _route_plain(s)


def work(c):
    if c["op"] == "linear":
        size, m = 2, 2 if c["gated"] else 1
        out = 4 if c["out"] == "f32" else 2
        byte = size * (c["t"] * c["k"] + m * c["n"] * c["k"]) + out * c["t"] * c["n"] * (2 if c["residual"] else 1)
        return {"bytes": byte + (4 * c["n"] * m if c["bias"] else 0), "flops": 2 * c["t"] * c["k"] * c["n"] * m}
    size = 2 if c["dtype"] == "bf16" else 4
    # per logit: a score (about 8 operations) and a comparison for each choice made
    return {"bytes": c["t"] * (size * c["e"] + 8 * c["top"]) + (4 * c["e"] if c["bias"] else 0),
            "flops": c["t"] * c["e"] * (8 + c["top"])}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "linear":
        x = s["x"].to(torch.float64)

        def product(w, b):
            y = torch.einsum("tk,nk->tn", x, w.to(torch.float64))
            return y if b is None else y.add_(b.to(torch.float64))

        y = product(s["w"], s["bias"])
        if case["act"] == "silu":
            y = torch.sigmoid(y) * y
        elif case["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        elif case["act"] == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        elif case["act"] == "relu":
            y = torch.relu(y)
        if case["gated"]:
            y = y * product(s["wu"], s["bias_u"])
        return y if s["residual"] is None else y + s["residual"].to(torch.float64)
    import numpy as np
    logits = s["logits"].double().cpu().numpy()
    t, e = logits.shape
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + np.exp(-logits))
    else:
        top = logits.max(1)[:, None]
        score = np.exp(logits - top - np.log(np.exp(logits - top).sum(1))[:, None])
    value = score if s["bias"] is None else score + s["bias"].double().cpu().numpy()[None]
    per = e // case["groups"]
    part = np.sort(value.reshape(t, case["groups"], per), axis=2)
    rank = part[..., -1] + (part[..., -2] if case["group_score"] == "top2" and per > 1 else 0.0)
    place = np.argsort(np.argsort(-rank, axis=1, kind="stable"), axis=1)
    outside = np.repeat(place >= case["keep"], per, axis=1)
    idx = np.lexsort((-value, outside), axis=1)[:, :case["top"]]
    w = np.take_along_axis(score, idx, 1)
    if case["renorm"]:
        w /= w.sum(1)[:, None]
    return idx.astype(np.int32), w * case["scale"]
