"""Operators around the ternary product, as measured cases.

Three kinds of call are listed:

  quantize  a matrix to microscaled 4-bit floats (e2m1 values, one power-of-two
            scale per 32 along a row) and back to the values that it stands for
  linear    Y = X . W^T with W held in that form and X in 16 bits
  linear4   the same with X quantised to that form first, within the call
  moe       a mixture-of-experts layer with ternary experts, from the router's
            logits to the summed outputs, for a few tokens

With ``own`` false every call is computed from elementary torch operations in
32 bits, rounded once at the end; with ``own`` true by the package's kernels.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_DEV = "cuda"


# --- cases -------------------------------------------------------------------

def listed():
    return [
        # one token's activations on their way into a 4-bit product: launch latency
        dict(name="quantize_token", kind="quantize", M=1, K=5120, x="bf16"),
        # a whole FFN weight matrix converted from its fp32 master copy
        dict(name="quantize_weights", kind="quantize", M=17408, K=5120, x="f32"),
        # attention projection of a single decoded token
        dict(name="linear_one_token", kind="linear", M=1, N=5120, K=5120, x="bf16", y="bf16"),
        # FFN up projection of four sequences decoded together
        dict(name="linear_four_tokens", kind="linear", M=4, N=17408, K=5120, x="bf16", y="bf16"),
        # FFN down projection, sixteen sequences, fp16 activations
        dict(name="linear_sixteen_tokens", kind="linear", M=16, N=5120, K=17408, x="f16", y="f16"),
        # a ragged batch through odd sizes: K ends inside a 128- and a 256-wide tile
        dict(name="linear_ragged", kind="linear", M=37, N=1001, K=1056, x="bf16", y="f32"),
        # fused query, key and value projection of a prompt
        dict(name="linear_prompt", kind="linear", M=2048, N=7168, K=5120, x="bf16", y="bf16"),
        # FFN up projection of a prompt with 4-bit activations
        dict(name="linear4_prompt", kind="linear4", M=2048, N=17408, K=5120, x="bf16", y="bf16"),
        # a ragged batch with 4-bit activations
        dict(name="linear4_ragged", kind="linear4", M=130, N=1111, K=2080, x="f16", y="f16"),
        # one decoded token through a layer of many small experts
        dict(name="moe_one_token", kind="moe", T=1, E=64, top_k=8, H=2048, F=1024, renorm=True, pad=0, x="bf16"),
        # four decoded tokens through a layer of few large experts
        dict(name="moe_four_tokens", kind="moe", T=4, E=8, top_k=2, H=5120, F=2048, renorm=False, pad=0, x="f16"),
        # a padded decode batch: the last tokens are padding (no expert is open to them)
        dict(name="moe_batch", kind="moe", T=32, E=64, top_k=8, H=2048, F=1024, renorm=True, pad=3, x="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quantize", "linear", "linear", "linear4", "moe", "moe"])
    if kind == "quantize":
        K = 32 * _log(rng, 1, 544)
        M = max(1, min(_log(rng, 1, 17408), 17408 * 5120 // K))
        return dict(kind=kind, M=M, K=K, x=rng.choice(["bf16", "f16", "f32"]))
    if kind in ("linear", "linear4"):
        K = 32 * _log(rng, 2, 544)
        N = _log(rng, 16, 17408)
        M = _log(rng, 1, 2048) if rng.random() < 0.5 else rng.randint(1, 16)
        M = max(1, min(M, (2048 * 7168 if kind == "linear" else 2048 * 17408) * 5120 // (N * K)))
        x = rng.choice(["bf16", "f16"])
        return dict(kind=kind, M=M, N=N, K=K, x=x, y=rng.choice([x, "f32"]))
    E = rng.randint(4, 128)
    H = 128 * _log(rng, 2, 40)
    F = 128 * _log(rng, 1, 16)
    E = max(2, min(E, 64 * 2048 * 1024 // (H * F)))
    return dict(kind=kind, T=_log(rng, 1, 64), E=E, top_k=rng.randint(1, min(8, E)), H=H, F=F,
                renorm=rng.random() < 0.5, pad=0, x=rng.choice(["bf16", "f16"]))


# --- inputs ------------------------------------------------------------------

def _generator(seed, stream):
    return torch.Generator(device=_DEV).manual_seed(seed * 16 + stream)


def _activations(shape, dtype, gen):
    """Normed activations with the rare large channels that decoders have."""
    x = torch.randn(shape, generator=gen, device=_DEV)
    big = torch.rand(shape, generator=gen, device=_DEV) < 0.01
    return torch.where(big, x * 8.0, x).to(dtype)


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
    dt = _DT[case["x"]]
    if kind == "quantize":
        if case["x"] == "f32":   # weights; otherwise activations
            s["x"] = torch.randn((case["M"], case["K"]), generator=_generator(seed, 0), device=_DEV) * 0.02
        else:
            s["x"] = _activations((case["M"], case["K"]), dt, _generator(seed, 0))
    elif kind in ("linear", "linear4"):
        s["x"] = _activations((case["M"], case["K"]), dt, _generator(seed, 0))
        w = torch.randn((case["N"], case["K"]), generator=_generator(seed, 1), device=_DEV) * 0.02
        s["codes"], s["exps"] = _quantize(w)
    else:
        T, E, H, F = case["T"], case["E"], case["H"], case["F"]
        s["x"] = torch.randn((T, H), generator=_generator(seed, 0), device=_DEV).to(dt)
        s["logits"] = torch.randn((T, E), generator=_generator(seed, 1), device=_DEV) * 1.5
        if case["pad"]:
            s["logits"][T - case["pad"]:] = -math.inf
        s["gate_up"] = _ternary((E, 2 * F, H // 4), _generator(seed, 2))
        s["gate_up_scales"] = _block_scales((E, 2 * F, H // 128), _generator(seed, 3))
        s["down"] = _ternary((E, H, F // 4), _generator(seed, 4))
        s["down_scales"] = _block_scales((E, H, F // 128), _generator(seed, 5))
    return s


# --- plain forms ---------------------------------------------------------------

def _quantize(x):
    """codes [M, K/2] (low nibble first) and biased exponents [M, K/32].

    The scale is 2^(floor(log2 of the largest magnitude) - 2), at least 2^-127;
    an element is rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 times the
    scale, ties to the even code, what lies above 6 to 6.
    """
    M, K = x.shape
    v = x.float().reshape(M, K // 32, 32)
    a = v.abs()
    field = a.amax(-1).contiguous().view(torch.int32) >> 23
    exps = (field - 2).clamp_(min=0)
    # a * 2^(127 - exps), a power of two that is exact in fp32
    a = a * ((254 - exps) << 23).view(torch.float32).unsqueeze(-1)
    code = torch.zeros_like(a, dtype=torch.uint8)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True),
                       (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= border) if up else (a > border)
    code |= torch.signbit(v).to(torch.uint8) << 3
    code = code.reshape(M, K // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), exps.to(torch.uint8)


def _values(codes, exps):
    """fp32 values of a quantised matrix."""
    N, half = codes.shape
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), dim=-1).to(torch.int32)
    e = exps.to(torch.int32)
    # 2^(e - 127); the field of an fp32 holds all but 2^-127
    scale = torch.where(e > 0, (e << 23).view(torch.float32), 2.0 ** -127)
    return (table[both].reshape(N, half * 2 // 32, 32) * scale.unsqueeze(-1)).reshape(N, 2 * half)


def _dense(packed, scales):
    """fp32 values of a ternary matrix [N, K/4] with scales [N, K/128]."""
    N, quarter = packed.shape
    c = torch.stack([(packed >> (2 * i)) & 3 for i in range(4)], dim=-1)
    t = (c == 1).float() - (c == 2).float()
    return (t.reshape(N, quarter * 4 // 128, 128) * scales.float().unsqueeze(-1)).reshape(N, quarter * 4)


def _route(logits, top_k, renorm):
    """Routing weights [T, E], zero where an expert is not taken."""
    logits = logits.float()
    order = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :top_k]
    taken = torch.zeros_like(logits).scatter_(1, order, 1.0)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    w = p * taken
    total = (w if renorm else p).sum(-1, keepdim=True)
    return torch.where(total > 0, w / total, 0.0)


def _moe(s):
    c = s["case"]
    F = c["F"]
    x = s["x"].float()
    w = _route(s["logits"], c["top_k"], c["renorm"])
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
        if kind == "quantize":
            codes, exps = tern.mx_quantize(state["x"])
            return tern.mx_dequant(codes, exps, out_dtype=torch.bfloat16)
        if kind == "linear":
            return tern.mx_matmul(state["x"], state["codes"], state["exps"], out_dtype=_DT[c["y"]])
        if kind == "linear4":
            xc, xe = tern.mx_quantize(state["x"])
            return tern.mx_matmul_mx(xc, xe, state["codes"], state["exps"], out_dtype=_DT[c["y"]])
        return tern.moe(state["x"], state["logits"], state["gate_up"], state["gate_up_scales"], state["down"],
                        state["down_scales"], top_k=c["top_k"], renormalize=c["renorm"])
    if kind == "quantize":
        return _values(*_quantize(state["x"])).to(torch.bfloat16)   # exact: two significant bits
    if kind == "linear":
        return (state["x"].float() @ _values(state["codes"], state["exps"]).t()).to(_DT[c["y"]])
    if kind == "linear4":
        x = _values(*_quantize(state["x"]))
        return (x @ _values(state["codes"], state["exps"]).t()).to(_DT[c["y"]])
    return _moe(state)


# --- what a pass cannot do without ----------------------------------------------

def work(case):
    kind = case["kind"]
    if kind == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": n * _BYTES[case["x"]] + n // 2 + n // 32 + 2 * n, "flops": 0}
    if kind in ("linear", "linear4"):
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": N * K // 2 + N * K // 32 + M * K * _BYTES[case["x"]] + M * N * _BYTES[case["y"]],
                "flops": 2 * M * N * K}
    T, E, k, H, F = (case[n] for n in ("T", "E", "top_k", "H", "F"))
    live = T - case["pad"]
    # every opened expert once: its expected number under even routing
    opened = E * (1.0 - (1.0 - k / E) ** live)
    per = 3 * H * F // 4 + 2 * (3 * H * F // 128)
    return {"bytes": int(opened * per) + 2 * T * H * _BYTES[case["x"]] + 4 * T * E,
            "flops": 2 * live * k * 3 * H * F}


# --- the definitions in 64 bits -------------------------------------------------

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_quantized(x):
    """Values of x after quantisation, from the definition: the nearest grid point, ties to the even one."""
    M, K = x.shape
    out = torch.empty((M, K), dtype=torch.float64, device=x.device)
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    for r in range(0, M, 1024):
        v = x[r:r + 1024].double().reshape(-1, K // 32, 32)
        _, e = torch.frexp(v.abs().amax(-1, keepdim=True))   # magnitude in [2^(e-1), 2^e)
        e = torch.where(v.abs().amax(-1, keepdim=True) > 0, e - 3, -127).clamp(min=-127)
        a = torch.ldexp(v.abs(), -e)
        hi = torch.searchsorted(grid, a.clamp(max=6.0).contiguous())   # first grid point >= a
        lo = (hi - 1).clamp(min=0)
        up, down = grid[hi] - a.clamp(max=6.0), a.clamp(max=6.0) - grid[lo]
        pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        out[r:r + 1024] = (torch.ldexp(grid[pick], e) * torch.where(v < 0, -1.0, 1.0)).reshape(-1, K)
    return out


def _exact_values(codes, exps):
    N, half = codes.shape
    out = torch.empty((N, half, 2), dtype=torch.float64, device=codes.device)
    for i in range(2):
        c = ((codes >> (4 * i)) & 15).long()
        m, e = c & 1, (c >> 1) & 3
        mag = torch.where(e > 0, (2 + m).double() * torch.pow(2.0, (e - 2).double()), m.double() * 0.5)
        out[..., i] = torch.where(c >= 8, -mag, mag)
    scale = torch.pow(2.0, exps.double() - 127.0)
    return (out.reshape(N, half * 2 // 32, 32) * scale.unsqueeze(-1)).reshape(N, half * 2)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantize":
        return _exact_quantized(s["x"])
    if kind in ("linear", "linear4"):
        x = s["x"].double() if kind == "linear" else _exact_quantized(s["x"])
        return x @ _exact_values(s["codes"], s["exps"]).t()
    T, E, k, H, F = (case[n] for n in ("T", "E", "top_k", "H", "F"))
    logits = s["logits"].double()
    # rank of an expert: how many come before it (greater, or equal with a lower index)
    before = (logits[:, None, :] > logits[:, :, None]) | (
        (logits[:, None, :] == logits[:, :, None])
        & (torch.arange(E, device=_DEV)[None, None, :] < torch.arange(E, device=_DEV)[None, :, None]))
    chosen = (before.sum(-1) < k) & (logits > -math.inf)
    kept = chosen if case["renorm"] else logits > -math.inf
    norm = torch.logsumexp(torch.where(kept, logits, -math.inf), dim=-1, keepdim=True)
    weight = torch.where(chosen, torch.exp(logits - torch.where(norm == -math.inf, 0.0, norm)), 0.0)
    x = s["x"].double()
    y = torch.zeros((T, H), dtype=torch.float64, device=_DEV)
    value = torch.tensor([0.0, 1.0, -1.0, 0.0], dtype=torch.float64, device=_DEV)
    for e in range(E):
        mats = []
        for p, sc in ((s["gate_up"][e], s["gate_up_scales"][e]), (s["down"][e], s["down_scales"][e])):
            t = torch.empty((p.shape[0], p.shape[1], 4), dtype=torch.float64, device=_DEV)
            for i in range(4):
                t[..., i] = value[((p.int() // 4 ** i) % 4).long()]
            mats.append(t.reshape(p.shape[0], -1) * sc.double().repeat_interleave(128, dim=1))
        gu = x @ mats[0].t()
        h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        y += weight[:, e:e + 1] * (h @ mats[1].t())
    return y
