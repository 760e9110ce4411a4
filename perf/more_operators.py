"""Operators on either side of the ternary products, as measured cases.

Five kinds of call are listed:

  norm      root-mean-square norm of a decoder's residual stream, with the
            addition to that stream where there is one, in 16 bits
  norm8     the same with 8-bit outputs and their scales, read back to the
            values that they stand for
  linear8   Y = X . (T*S)^T with X in 8 bits with scales and ternary weights
  route     a router's logits to the experts that its tokens take: softmax or
            sigmoid scores, a bias for balance, groups of experts, top-k
  experts   the same routing, and the mixture of ternary experts that it is for

With ``own`` false every call is computed from elementary torch operations in
32 bits (64 where a code or a choice hangs on the last bit), rounded once at
the end; with ``own`` true by the package's kernels.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_DEV = "cuda"
_EPS = 1e-6


# --- cases -------------------------------------------------------------------

def listed():
    return [
        # norms of the query and key heads of a prompt: many short rows, no residual
        dict(name="norm_heads", kind="norm", M=32768, K=128, x="bf16", r="", w="bf16"),
        # the norm before a prompt's projections, residual stream in 16 bits
        dict(name="norm_prompt", kind="norm", M=2048, K=5120, x="bf16", r="bf16", w="bf16"),
        # one decoded token on its way into an 8-bit product, a scale for the token: launch latency
        dict(name="norm8_one_token", kind="norm8", M=1, K=5120, x="bf16", r="bf16", w="bf16", group=0),
        # a ragged batch before a wide down projection, residual stream in 32 bits, a scale per 128
        dict(name="norm8_ragged", kind="norm8", M=333, K=17408, x="f16", r="f32", w="f32", group=128),
        # attention projection of a single decoded token
        dict(name="linear8_one_token", kind="linear8", M=1, N=5120, K=5120, group=0, y="bf16"),
        # FFN down projection of sixteen sequences decoded together
        dict(name="linear8_sixteen_tokens", kind="linear8", M=16, N=5120, K=17408, group=0, y="bf16"),
        # a ragged batch through odd sizes, a scale per 128 activations
        dict(name="linear8_ragged", kind="linear8", M=37, N=1001, K=1152, group=128, y="f32"),
        # FFN up projection of a prompt
        dict(name="linear8_prompt", kind="linear8", M=2048, N=17408, K=5120, group=0, y="bf16"),
        # one decoded token, sigmoid scores with a balancing bias, 4 of 8 groups: launch latency
        dict(name="route_one_token", kind="route", T=1, E=256, top_k=8, score="sigmoid", bias=True, groups=8, keep=4,
             best=2, renorm=True, scale=2.5, l="f32"),
        # the tokens of a long prompt, softmax scores, one group
        dict(name="route_prompt", kind="route", T=8192, E=128, top_k=8, score="softmax", bias=False, groups=1, keep=1,
             best=1, renorm=True, scale=1.0, l="bf16"),
        # one decoded token through a layer of many small experts, groups and bias
        dict(name="experts_one_token", kind="experts", T=1, E=64, top_k=6, score="sigmoid", bias=True, groups=4, keep=2,
             best=2, renorm=True, scale=2.5, l="f32", H=2048, F=1024, x="bf16"),
        # a decode batch through the same layer
        dict(name="experts_batch", kind="experts", T=24, E=64, top_k=6, score="sigmoid", bias=True, groups=4, keep=2,
             best=2, renorm=True, scale=2.5, l="f32", H=2048, F=1024, x="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_router(rng, case, most):
    groups = rng.choice([1, 1, 2, 4, 8])
    per = max(2, _log(rng, 4, most) // groups)
    case.update(E=groups * per, groups=groups, keep=rng.randint(1, groups), bias=rng.random() < 0.6,
                score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.7, best=rng.choice([1, 2]),
                scale=rng.choice([1.0, 2.5]), l=rng.choice(["f32", "bf16", "f16"]))
    case["top_k"] = rng.randint(1, min(10, case["keep"] * per))
    return case


def draw(rng):
    kind = rng.choice(["norm", "norm8", "linear8", "linear8", "route", "experts"])
    if kind in ("norm", "norm8"):
        group = rng.choice([0, 128]) if kind == "norm8" else 0
        K = 128 * _log(rng, 1, 136) if group else _log(rng, 64, 17408)
        M = max(1, min(_log(rng, 1, 32768), 333 * 17408 // K))
        x = rng.choice(["bf16", "f16"])
        case = dict(kind=kind, M=M, K=K, x=x, r=rng.choice(["", x, "f32"]), w=rng.choice([x, "f32"]))
        if kind == "norm8":
            case["group"] = group
        return case
    if kind == "linear8":
        K = 128 * _log(rng, 1, 136)
        N = _log(rng, 16, 17408)
        M = _log(rng, 1, 2048) if rng.random() < 0.5 else rng.randint(1, 16)
        M = max(1, min(M, 2048 * 17408 * 5120 // (N * K)))
        return dict(kind=kind, M=M, N=N, K=K, group=rng.choice([0, 128]), y=rng.choice(["bf16", "f16", "f32"]))
    if kind == "route":
        return _draw_router(rng, dict(kind=kind, T=_log(rng, 1, 4096)), 256)
    H = 128 * _log(rng, 2, 40)
    F = 128 * _log(rng, 1, 16)
    most = max(8, min(64, 64 * 2048 * 1024 // (H * F)))
    return _draw_router(rng, dict(kind=kind, T=_log(rng, 1, 24), H=H, F=F, x=rng.choice(["bf16", "f16"])), most)


# --- inputs ------------------------------------------------------------------

def _generator(seed, stream):
    return torch.Generator(device=_DEV).manual_seed(seed * 16 + stream)


def _activations(shape, gen):
    """Values with the rare large channels that decoders have."""
    x = torch.randn(shape, generator=gen, device=_DEV)
    big = torch.rand(shape, generator=gen, device=_DEV) < 0.01
    return torch.where(big, x * 8.0, x)


def _ternary(shape, gen):
    """Packed codes: 40% zeros, 30% of either sign, four to a byte."""
    out = None
    for i in range(4):
        r = torch.randint(0, 10, shape, generator=gen, device=_DEV, dtype=torch.uint8)
        c = torch.where(r < 4, 0, torch.where(r < 7, 1, 2)).to(torch.uint8)
        out = c if out is None else out | (c << (2 * i))
    return out


def _block_scales(shape, gen):
    """Log-uniform over [1e-3, 1e-1]."""
    u = torch.rand(shape, generator=gen, device=_DEV)
    return torch.exp(u * math.log(100.0) + math.log(1e-3)).half()


def prepare(case, seed):
    s = dict(case=dict(case))
    kind = case["kind"]
    if kind in ("norm", "norm8"):
        M, K = case["M"], case["K"]
        s["x"] = _activations((M, K), _generator(seed, 0)).to(_DT[case["x"]])
        s["r"] = (_activations((M, K), _generator(seed, 1)) * 4.0).to(_DT[case["r"]]) if case["r"] else None
        s["w"] = (1.0 + 0.2 * torch.randn((K,), generator=_generator(seed, 2), device=_DEV)).to(_DT[case["w"]])
    elif kind == "linear8":
        M, N, K = case["M"], case["N"], case["K"]
        s["codes"], scales = _codes(_activations((M, K), _generator(seed, 0)), case["group"])
        s["scales"] = scales / 127.0
        s["packed"] = _ternary((N, K // 4), _generator(seed, 1))
        s["weight_scales"] = _block_scales((N, K // 128), _generator(seed, 2))
    else:
        T, E = case["T"], case["E"]
        s["logits"] = (torch.randn((T, E), generator=_generator(seed, 0), device=_DEV) * 1.5).to(_DT[case["l"]])
        s["bias"] = 0.1 * torch.randn((E,), generator=_generator(seed, 1), device=_DEV) if case["bias"] else None
        if kind == "experts":
            H, F = case["H"], case["F"]
            s["x"] = torch.randn((T, H), generator=_generator(seed, 2), device=_DEV).to(_DT[case["x"]])
            s["gate_up"] = _ternary((E, 2 * F, H // 4), _generator(seed, 3))
            s["gate_up_scales"] = _block_scales((E, 2 * F, H // 128), _generator(seed, 4))
            s["down"] = _ternary((E, H, F // 4), _generator(seed, 5))
            s["down_scales"] = _block_scales((E, H, F // 128), _generator(seed, 6))
    return s


# --- plain forms ---------------------------------------------------------------

def _codes(v, group):
    """int8 codes of v [M,K] and the largest magnitude (fp32) of each row, or of each `group` of a row.

    A code is 127 v / largest, rounded to nearest, ties to even: in 64 bits, as it hangs on the last bit.
    """
    M, K = v.shape
    width = group if group else K
    b = v.reshape(M, K // width, width)
    top = b.abs().amax(-1).float()
    q = torch.round(127.0 * b.double() / torch.where(top > 0, top, 1.0).double().unsqueeze(-1))
    return q.to(torch.int8).reshape(M, K), top


def _norm(s):
    c = s["case"]
    x, w = s["x"].float(), s["w"].float()
    h = None
    if s["r"] is not None:
        h = (x + s["r"].float()).to(s["r"].dtype)   # what the stream holds from here on
        x = h.float()
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    if c["kind"] == "norm":
        y = (x * rstd * w).to(s["x"].dtype)
    else:
        # the row's factor does not change which codes its values get
        q, top = _codes(x.double() * w.double(), c["group"])
        M, K = q.shape
        scales = top * rstd / 127.0
        y = (q.float().reshape(M, scales.shape[1], -1) * scales.unsqueeze(-1)).reshape(M, K)
    return y if h is None else (y, h)


def _dense(packed, scales):
    """fp32 values of a ternary matrix [N, K/4] with scales [N, K/128]."""
    N, quarter = packed.shape
    c = torch.stack([(packed >> (2 * i)) & 3 for i in range(4)], dim=-1)
    t = (c == 1).float() - (c == 2).float()
    return (t.reshape(N, quarter * 4 // 128, 128) * scales.float().unsqueeze(-1)).reshape(N, quarter * 4)


def _route(s):
    """Experts [T, top_k] in the order of their scores, and their weights."""
    c = s["case"]
    logits = s["logits"].double()
    T, E = logits.shape
    if c["score"] == "softmax":
        p = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = p / p.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    choice = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        each = choice.reshape(T, c["groups"], -1)
        best = torch.sort(each, dim=-1, descending=True).values[..., :c["best"]].sum(-1)
        kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        open_ = torch.zeros_like(best).scatter_(1, kept, 1.0) > 0
        choice = torch.where(open_.unsqueeze(-1), each, -math.inf).reshape(T, E)
    ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = torch.gather(score, 1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _experts(s):
    c = s["case"]
    F = c["F"]
    x = s["x"].float()
    ids, weights = _route(s)
    w = torch.zeros((c["T"], c["E"]), device=x.device).scatter_(1, ids.long(), weights)
    y = torch.zeros_like(x)
    for e in range(c["E"]):
        gu = x @ _dense(s["gate_up"][e], s["gate_up_scales"][e]).t()
        g, u = gu[:, :F], gu[:, F:]
        h = g / (1.0 + torch.exp(-g)) * u
        y = y + w[:, e:e + 1] * (h @ _dense(s["down"][e], s["down_scales"][e]).t())
    return y.to(s["x"].dtype)


def run(state):
    c = state["case"]
    kind = c["kind"]
    if own:
        import ternary_weight_matmul_amd as tern
        if kind == "norm":
            return tern.rms_norm(state["x"], state["w"], eps=_EPS, residual=state["r"])
        if kind == "norm8":
            codes, scales, *h = tern.rms_norm_q8(state["x"], state["w"], eps=_EPS, residual=state["r"],
                                                 group=c["group"])
            y = tern.q8_dequant(codes, scales, out_dtype=torch.float32)
            return (y, *h) if h else y
        if kind == "linear8":
            return tern.matmul_q8(state["codes"], state["scales"], state["packed"], state["weight_scales"],
                                  out_dtype=_DT[c["y"]])
        ids, weights = tern.moe_route(state["logits"], c["top_k"], score=c["score"], bias=state["bias"],
                                      groups=c["groups"], keep_groups=c["keep"], group_best=c["best"],
                                      renormalize=c["renorm"], scale=c["scale"])
        if kind == "route":
            return ids, weights
        return tern.moe_routed(state["x"], ids, weights, state["gate_up"], state["gate_up_scales"], state["down"],
                               state["down_scales"])
    if kind in ("norm", "norm8"):
        return _norm(state)
    if kind == "linear8":
        q, scales = state["codes"].float(), state["scales"]
        x = (q.reshape(c["M"], scales.shape[1], -1) * scales.unsqueeze(-1)).reshape(c["M"], c["K"])
        return (x @ _dense(state["packed"], state["weight_scales"]).t()).to(_DT[c["y"]])
    return _route(state) if kind == "route" else _experts(state)


# --- what a pass cannot do without ----------------------------------------------

def work(case):
    kind = case["kind"]
    if kind in ("norm", "norm8"):
        M, K = case["M"], case["K"]
        r = 2 * _BYTES[case["r"]] if case["r"] else 0
        y = _BYTES[case["x"]] if kind == "norm" else 4
        return {"bytes": M * K * (_BYTES[case["x"]] + r + y) + K * _BYTES[case["w"]], "flops": 4 * M * K}
    if kind == "linear8":
        M, N, K = case["M"], case["N"], case["K"]
        xs = M * (K // 128 if case["group"] else 1) * 4
        return {"bytes": N * K // 4 + N * K // 64 + M * K + xs + M * N * _BYTES[case["y"]], "flops": 2 * M * N * K}
    T, E, k = case["T"], case["E"], case["top_k"]
    logits = T * E * _BYTES[case["l"]] + (4 * E if case["bias"] else 0)
    if kind == "route":
        return {"bytes": logits + 8 * T * k, "flops": 4 * T * E}
    H, F = case["H"], case["F"]
    # every opened expert once: its expected number under even routing
    opened = E * (1.0 - (1.0 - k / E) ** T)
    per = 3 * H * F // 4 + 2 * (3 * H * F // 128)
    return {"bytes": int(opened * per) + 2 * T * H * _BYTES[case["x"]] + logits, "flops": 2 * T * k * 3 * H * F}


# --- the definitions in 64 bits -------------------------------------------------

def _exact_norm(s):
    c = s["case"]
    M, K = s["x"].shape
    x, w = s["x"].double(), s["w"].double()
    h = None
    if s["r"] is not None:
        h = (x + s["r"].double()).to(s["r"].dtype).double()
        x = h
    root = torch.sqrt(torch.linalg.vecdot(x, x).unsqueeze(-1) / K + _EPS)
    v = x * w
    if c["kind"] == "norm":
        y = v / root
    else:
        blocks = v.reshape(M, -1, c["group"] or K)
        top = blocks.abs().max(dim=-1, keepdim=True).values.float().double()
        scaled = torch.where(top > 0, 127.0 * blocks / top, 0.0)
        low = torch.floor(scaled)
        over = scaled - low
        q = low + ((over > 0.5) | ((over == 0.5) & (torch.remainder(low, 2.0) == 1.0))).double()
        y = (q * top / 127.0).reshape(M, K) / root
    return y if h is None else (y, h)


def _exact_dense(packed, scales):
    value = torch.tensor([0.0, 1.0, -1.0, 0.0], dtype=torch.float64, device=_DEV)
    t = torch.empty((*packed.shape, 4), dtype=torch.float64, device=_DEV)
    for i in range(4):
        t[..., i] = value[((packed.int() // 4 ** i) % 4).long()]
    return t.reshape(packed.shape[0], -1) * scales.double().repeat_interleave(128, dim=1)


def _ranks(v):
    """How many of a row come before each: greater, or equal with a lower index."""
    at = torch.arange(v.shape[-1], device=v.device)
    a, b = v.unsqueeze(-1), v.unsqueeze(-2)   # a: the one ranked, b: the others
    return ((b > a) | ((b == a) & (at < at.unsqueeze(-1)))).sum(-1)


def _exact_route(s):
    c = s["case"]
    E, k = c["E"], c["top_k"]
    per = E // c["groups"]
    all_ids, all_w = [], []
    for logits in s["logits"].double().split(512):
        score = torch.softmax(logits, -1) if c["score"] == "softmax" else torch.sigmoid(logits)
        choice = score + (s["bias"].double() if s["bias"] is not None else 0.0)
        in_groups = choice.reshape(-1, c["groups"], per)
        total = torch.where(_ranks(in_groups) < c["best"], in_groups, 0.0).sum(-1)
        kept = (_ranks(total) < c["keep"]).repeat_interleave(per, dim=1)
        if c["groups"] > 1:
            choice = torch.where(kept, choice, -math.inf)
        rank = _ranks(choice)
        ids = torch.argsort(rank, dim=-1)[:, :k]
        w = score.gather(1, ids)
        all_ids.append(ids)
        all_w.append(w / (w.sum(-1, keepdim=True) if c["renorm"] else 1.0) * c["scale"])
    return torch.cat(all_ids).to(torch.int32), torch.cat(all_w)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("norm", "norm8"):
        return _exact_norm(s)
    if kind == "linear8":
        width = case["group"] or case["K"]
        x = s["codes"].double() * s["scales"].double().repeat_interleave(width, dim=1)
        return x @ _exact_dense(s["packed"], s["weight_scales"]).t()
    ids, weights = _exact_route(s)
    if kind == "route":
        return ids, weights
    x = s["x"].double()
    F = case["F"]
    y = torch.zeros_like(x)
    for e in range(case["E"]):
        rows, place = torch.nonzero(ids == e, as_tuple=True)
        if rows.numel() == 0:
            continue
        gu = x[rows] @ _exact_dense(s["gate_up"][e], s["gate_up_scales"][e]).t()
        h = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
        y[rows] += weights[rows, place].unsqueeze(-1) * (h @ _exact_dense(s["down"][e], s["down_scales"][e]).t())
    return y
