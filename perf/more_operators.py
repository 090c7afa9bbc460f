"""Measured operators of a mixture-of-experts feed-forward block: routing of
tokens to experts, the experts' products on MXFP4 weights, and the norms around
a block fused with its gate and residual scale.

Routing. l = logits with NaN as -inf and +inf as the largest float32; the score
s is softmax(l) or sigmoid(l), 0 where l = -inf. Experts are chosen by c = l, or
with a bias by c = float32(s + bias) (-inf where l is), s in 64 bits. With
groups of equal size, those with the highest group scores stay and the others'
c become -inf; a group's score is its highest c, with a bias the sum of its two
highest (one of -inf adds nothing). The k highest c are taken, ties to the lower
index; their weights are s (0 at c = -inf), divided by their sum if asked, times
a factor.

Experts. For each pair of a token and one of its experts:
  a = silu(Wg x^) * (Wu x^),  o = Wd h^,  y = bf16(sum over pairs of w o)
with x^ the microscaled quantization of x, h^ that of bf16(a), and MXFP4
weights, Wg above Wu in one operand. Pairs whose expert is outside 0 .. E-1 are
skipped.

Block norm. n = x, or its RMS norm times a gain; h = alpha residual + gate n,
rounded to the residual's type; y = bf16(norm(h) gain (1 + scale) + shift), the
norm RMS or layer; MXFP8 codes of y in a slab.

Formats as in operators.py: groups of 32 along K with one scale 2**e, E4M3 or
E2M1 elements. MXFP4 weights lie in one slab for each expert: codes uint8
[E, ceil(K/128), R/16, 4, 16, 16], scales uint8 [E, ceil(K/128), R, 4], R = rows
rounded up to 256; MXFP8 slabs are [K/64, R, 64] and [K/64, R, 2].

`own = False` computes each operator in elementary torch operations; `own =
True` makes the library's calls on the same data.
"""

import math

import torch

own = False

DEV = "cuda"
GROUP = 32
HIDDEN, VIDEO = 5120, 75348  # the transformer's hidden size and video tokens
EPS = 1e-6
F32_MAX = torch.finfo(torch.float32).max


def listed():
    return [
        # One decoded token, a step of a serving batch and a long prompt.
        {"name": "route_decode", "op": "route", "T": 1, "E": 128, "k": 8, "scores": "softmax", "bias": False,
         "groups": 1, "top": 1, "dtype": "f32"},
        {"name": "route_batch", "op": "route", "T": 509, "E": 64, "k": 6, "scores": "softmax", "bias": False,
         "groups": 8, "top": 3, "dtype": "bf16"},
        {"name": "route_prompt", "op": "route", "T": 32001, "E": 256, "k": 8, "scores": "sigmoid", "bias": True,
         "groups": 8, "top": 4, "dtype": "f32"},
        # One decoded token: the weights of its experts are all there is to read.
        {"name": "experts_decode", "op": "experts", "act": "fp8", "T": 1, "E": 64, "k": 8, "H": HIDDEN, "I": 2048},
        # Small serving batches: most experts have a few tokens.
        {"name": "experts_batch", "op": "experts", "act": "fp8", "T": 13, "E": 64, "k": 4, "H": 4096, "I": 1408},
        {"name": "experts_serve", "op": "experts", "act": "fp4", "T": 128, "E": 64, "k": 8, "H": 4096, "I": 1408},
        # Prompts: hundreds of tokens for each expert.
        {"name": "experts_prompt8", "op": "experts", "act": "fp8", "T": 4001, "E": 64, "k": 8, "H": 4096, "I": 2048},
        {"name": "experts_prompt4", "op": "experts", "act": "fp4", "T": 8192, "E": 32, "k": 4, "H": HIDDEN, "I": 2048},
        # A decoded token between two blocks of a language model (norms after
        # and before), a prompt with an fp32 residual stream, and the video
        # tokens of a diffusion transformer (gated residual, modulated layer norm).
        {"name": "norm_decode", "op": "norm", "M": 1, "K": HIDDEN, "res": "bf16", "post": True, "gate": "none",
         "kind": "rms", "mod": False},
        {"name": "norm_prompt", "op": "norm", "M": 509, "K": 4096, "res": "f32", "post": True, "gate": "vector",
         "kind": "rms", "mod": False},
        {"name": "norm_video", "op": "norm", "M": VIDEO, "K": HIDDEN, "res": "bf16", "post": False, "gate": "rows",
         "kind": "layer", "mod": True},
    ]


def _logint(rng, lo, hi, step):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "norm"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _logint(rng, 8 if groups > 1 else 16, 256 // groups, 1)
        top = rng.randint(1, groups)
        return {"op": op, "T": _logint(rng, 1, 30000, 1), "E": E, "k": rng.randint(1, min(8, top * (E // groups))),
                "scores": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "top": top, "dtype": rng.choice(["f32", "bf16"])}
    if op == "experts":
        E, H, I = _logint(rng, 4, 64, 1), _logint(rng, 512, 5120, 32), _logint(rng, 256, 2048, 32)
        return {"op": op, "act": rng.choice(["fp8", "fp4"]), "T": _logint(rng, 1, 4000, 1), "E": E,
                "k": rng.randint(1, min(8, E)), "H": H, "I": I}
    return {"op": op, "M": _logint(rng, 1, 40000, 1), "K": _logint(rng, 512, 8192, 64),
            "res": rng.choice(["bf16", "f32"]), "post": rng.random() < 0.5,
            "gate": rng.choice(["none", "vector", "rows"]), "kind": rng.choice(["rms", "layer"]),
            "mod": rng.random() < 0.5}


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (4 if case["dtype"] == "f32" else 2) + 8 * T * k + (4 * E if case["bias"] else 0),
                "flops": 10 * T * E}
    if case["op"] == "experts":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        used = E * (1.0 - (1.0 - k / E) ** T)  # experts with a token, were all as likely
        return {"bytes": int(used * 3 * I * H * 17 / 32) + 4 * T * H + 8 * T * k, "flops": 6 * T * k * I * H}
    M, K = case["M"], case["K"]
    es = 2 if case["res"] == "bf16" else 4
    vectors = K * 4 * ((case["post"]) + (case["gate"] != "none") + 1 + 2 * case["mod"])
    return {"bytes": M * K * (2 + 2 * es + 1) + M * K // 32 + vectors, "flops": 12 * M * K}


# ---------------------------------------------------------------------------
# Inputs.


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV)


def _activation(M, K, g):
    """N(0, 1) with one entry in a thousand 50 times larger, as activations have."""
    x = _randn((M, K), g)
    out = torch.rand((M, K), generator=g, device=DEV) < 1e-3
    return torch.where(out, 50.0 * x, x).to(torch.bfloat16)


def _expert_weights(E, rows, K, g):
    """The weights a program keeps: MXFP4 codes and scales, one slab an expert."""
    S, R = (K + 127) // 128, _rows(rows)
    q = torch.empty((E, S, R // 16, 4, 16, 16), dtype=torch.uint8, device=DEV)
    s = torch.empty((E, S, R, 4), dtype=torch.uint8, device=DEV)
    for e in range(E):
        q[e], s[e] = _pack4(*_quantize(0.02 * _randn((rows, K), g), "fp4"))
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": dict(case)}
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        # Some experts are more in demand than others.
        logits = 1.5 * _randn((T, E), g) + 0.5 * _randn((1, E), g)
        st["logits"] = logits if case["dtype"] == "f32" else logits.to(torch.bfloat16)
        st["bias"] = 0.05 * _randn((E,), g) if case["bias"] else None
    elif case["op"] == "experts":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        st["x"] = _activation(T, H, g)
        logits = 1.5 * _randn((T, E), g) + 0.5 * _randn((1, E), g)
        top, ids = torch.sort(logits, dim=1, descending=True)
        st["ids"] = ids[:, :k].to(torch.int32).contiguous()
        st["weights"] = torch.softmax(top[:, :k], dim=1).contiguous()
        st["up"] = _expert_weights(E, 2 * I, H, g)
        st["down"] = _expert_weights(E, H, I, g)
    else:
        M, K = case["M"], case["K"]
        st["x"] = _activation(M, K, g)
        r = 3.0 * _randn((M, K), g)
        st["residual"] = r.to(torch.bfloat16) if case["res"] == "bf16" else r
        st["post"] = 1.0 + 0.1 * _randn((K,), g) if case["post"] else None
        # One gate for all rows, or one for each of two samples of a batch.
        rows = 2 if M % 2 == 0 else 1
        st["gate"] = {"none": None, "vector": 0.5 + 0.1 * _randn((1, K), g),
                      "rows": 0.5 + 0.1 * _randn((rows, K), g)}[case["gate"]]
        st["gain"] = 1.0 + 0.1 * _randn((K,), g)
        st["scale"] = 0.1 * _randn((rows, K), g) if case["mod"] else None
        st["shift"] = 0.1 * _randn((rows, K), g) if case["mod"] else None
        st["alpha"] = 1.0 if case["kind"] == "layer" else 0.75
    return st


# ---------------------------------------------------------------------------
# Plain form.


def _rows(n):
    return (n + 255) // 256 * 256


def _pow2(e):
    """2**e as float32 for integer e in [-126, 127]."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantize(x, fmt):
    """Microscaled quantization of float32 [rows, K]: element values before
    the scale [rows, K/32, 32] and exponents e [rows, K/32]."""
    g = x.view(x.shape[0], -1, GROUP)
    amax = g.abs().amax(dim=-1)
    p = torch.frexp(amax).exponent.to(torch.int32) - 1
    e = torch.where(amax > 0, p - (2 if fmt == "fp4" else 8), torch.full_like(p, -127)).clamp(-127, 127)
    v = g * _pow2(-e)[..., None]
    if fmt == "fp8":
        return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).to(torch.float32), e
    a = v.abs()
    # E2M1 magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6: steps of 0.5, 1 and 2.
    r = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return torch.copysign(r.clamp(max=6.0), v), e


def _scaled(v, e):
    """Values of quantized data, float32 [rows, K]."""
    s = torch.where(e > -127, _pow2(e.clamp(min=-126)), torch.full_like(v[..., 0], 2.0**-127))
    return (v * s[..., None]).view(v.shape[0], -1)


def _pack4(v, e):
    rows, groups = e.shape
    S, R = (groups + 3) // 4, _rows(rows)
    a = v.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code |= torch.signbit(v).to(torch.uint8) << 3
    byte = (code[..., 0::2] | (code[..., 1::2] << 4)).view(rows, groups * 16)
    q = torch.zeros((R, S * 64), dtype=torch.uint8, device=v.device)
    q[:rows, : groups * 16] = byte
    q = q.view(R // 16, 16, S, 4, 16).permute(2, 0, 3, 1, 4).contiguous()
    s = torch.zeros((R, S * 4), dtype=torch.uint8, device=v.device)
    s[:rows, :groups] = (e + 127).to(torch.uint8)
    return q, s.view(R, S, 4).transpose(0, 1).contiguous()


def _pack8(v, e):
    rows, groups = e.shape
    S, R = groups // 2, _rows(rows)
    q = torch.zeros((S, R, 64), dtype=torch.uint8, device=v.device)
    q[:, :rows] = v.to(torch.float8_e4m3fn).view(torch.uint8).view(rows, S, 64).transpose(0, 1)
    s = torch.zeros((S, R, 2), dtype=torch.uint8, device=v.device)
    s[:, :rows] = (e + 127).to(torch.uint8).view(rows, S, 2).transpose(0, 1)
    return q, s


def _unpack4(q, s, rows, K):
    """Values of MXFP4 slabs [n, S, R/16, 4, 16, 16], float32 [n, rows, K]."""
    n = q.shape[0]
    b = q.permute(0, 2, 4, 1, 3, 5).reshape(n, q.shape[2] * 16, -1)[:, :rows, : K // 2]
    code = torch.stack((b & 15, b >> 4), dim=-1).view(n, rows, K).to(torch.int32)
    m = (code & 7).to(torch.float32)
    a = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    v = torch.where(code >= 8, -a, a).view(n, rows, K // GROUP, GROUP)
    e = s[:, :, :rows].transpose(1, 2).reshape(n, rows, -1)[:, :, : K // GROUP].to(torch.int32) - 127
    f = torch.where(e > -127, _pow2(e.clamp(min=-126)), torch.full_like(v[..., 0], 2.0**-127))
    return (v * f[..., None]).view(n, rows, K)


def _plain_route(st):
    c = st["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = st["logits"].to(torch.float32)
    l = torch.where(torch.isnan(l), torch.full_like(l, -math.inf), l).clamp(max=F32_MAX)
    live = l > -math.inf
    d = l.to(torch.float64)
    if c["scores"] == "softmax":
        p = torch.where(live, torch.exp(d - d.amax(dim=1, keepdim=True)), torch.zeros_like(d))
        s = p / p.sum(dim=1, keepdim=True).clamp(min=1e-300)
    else:
        s = 1.0 / (1.0 + torch.exp(-d))
    none = torch.full_like(l, -math.inf)
    key = l if st["bias"] is None else torch.where(live, (s + st["bias"].to(torch.float64)).to(torch.float32), none)
    if G > 1:
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values
        score = best[..., 0]
        if st["bias"] is not None and E // G > 1:
            score = score + torch.where(best[..., 1] > -math.inf, best[..., 1], torch.zeros_like(score))
        chosen = torch.sort(score, dim=1, descending=True, stable=True).indices[:, : c["top"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter(1, chosen, True)
        key = torch.where(kept.repeat_interleave(E // G, dim=1), key, none)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    w = torch.where(top > -math.inf, s.gather(1, ids), torch.zeros_like(s[:, :k]))
    total = w.sum(dim=1, keepdim=True)
    w = torch.where(total > 0, w / total, torch.zeros_like(w)) * 2.5
    return {"ids": ids.to(torch.int32), "weights": w.to(torch.float32)}


def _gated(v, I, act):
    """MX values of bf16(silu(gate) * up) for float32 [rows, 2 I]."""
    a = v[:, :I]
    a = a / (1.0 + torch.exp(-a)) * v[:, I:]
    return _scaled(*_quantize(a.to(torch.bfloat16).to(torch.float32), act))


def _plain_experts(st):
    c = st["case"]
    T, E, k, H, I = (c[n] for n in ("T", "E", "k", "H", "I"))
    x = _scaled(*_quantize(st["x"].to(torch.float32), c["act"]))
    ids, P = st["ids"].view(-1).to(torch.int64), T * k
    if P <= E:  # a few pairs: each with its expert's weights
        e = ids
        rows = x.repeat_interleave(k, dim=0)
        u = torch.bmm(_unpack4(st["up"][0][e], st["up"][1][e], 2 * I, H), rows[:, :, None])[:, :, 0]
        o = torch.bmm(_unpack4(st["down"][0][e], st["down"][1][e], H, I), _gated(u, I, c["act"])[:, :, None])[:, :, 0]
    else:  # the pairs sorted by expert, each expert's padded to the longest list
        order = torch.sort(ids, stable=True).indices
        counts = torch.bincount(ids, minlength=E)
        width = int(counts.max())
        sorted_ids = ids[order]
        place = sorted_ids * width + torch.arange(P, device=x.device) - (counts.cumsum(0) - counts)[sorted_ids]
        rows = torch.zeros((E * width, H), device=x.device)
        rows[place] = x[order // k]
        u = torch.bmm(rows.view(E, width, H), _unpack4(*st["up"], 2 * I, H).transpose(1, 2)).view(E * width, 2 * I)
        h = _gated(u, I, c["act"]).view(E, width, I)
        z = torch.bmm(h, _unpack4(*st["down"], H, I).transpose(1, 2)).view(E * width, H)
        o = torch.empty((P, H), device=x.device)
        o[order] = z[place]
    return (o.view(T, k, H) * st["weights"][..., None]).sum(dim=1).to(torch.bfloat16)


def _per_row(v, M):
    """A [n, K] vector set for M rows, float64 [M or 1, K]."""
    v = v.to(torch.float64)
    return v if v.shape[0] == 1 else v.repeat_interleave(M // v.shape[0], dim=0)


def _plain_norm(st):
    """Sums and products in 64 bits, since y is next rounded to few bits."""
    c, M = st["case"], st["case"]["M"]
    n = st["x"].to(torch.float64)
    if st["post"] is not None:
        n = n * (1.0 / torch.sqrt((n * n).mean(dim=-1, keepdim=True) + EPS)) * st["post"].to(torch.float64)
    if st["gate"] is not None:
        n = n * _per_row(st["gate"], M)
    h = (st["alpha"] * st["residual"].to(torch.float64) + n).to(torch.float32).to(st["residual"].dtype)
    d = h.to(torch.float64)
    if c["kind"] == "layer":
        d = d - d.mean(dim=-1, keepdim=True)
    y = d * (1.0 / torch.sqrt((d * d).mean(dim=-1, keepdim=True) + EPS)) * st["gain"].to(torch.float64)
    if st["scale"] is not None:
        y = y * (1.0 + _per_row(st["scale"], M)) + _per_row(st["shift"], M)
    y = y.to(torch.float32).to(torch.bfloat16)
    q, s = _pack8(*_quantize(y.to(torch.float32), "fp8"))
    return {"residual": h, "codes": q.view(torch.float8_e4m3fn), "scales": s.view(torch.float8_e8m0fnu)}


# ---------------------------------------------------------------------------
# The library's calls.


def _library(st):
    import mxfp8_w8a8_quantized_amd as mx

    c = st["case"]
    if c["op"] == "route":
        ids, w = mx.mx_route(st["logits"], c["k"], scores=c["scores"], bias=st["bias"], groups=c["groups"],
                             top_groups=c["top"], renorm=True, scale=2.5)
        return {"ids": ids, "weights": w}
    if c["op"] == "experts":
        up = mx.FP4Experts(*st["up"], 2 * c["I"], c["H"])
        down = mx.FP4Experts(*st["down"], c["H"], c["I"])
        return mx.mx_fp4_experts(st["x"], st["ids"], st["weights"], up, down, act=c["act"])
    slab, h = mx.mx_block_norm_slab(st["x"], st["residual"], post=st["post"] is not None, post_weight=st["post"],
                                    gate=st["gate"], residual_scale=st["alpha"], kind=c["kind"], weight=st["gain"],
                                    scale=st["scale"], shift=st["shift"], eps=EPS)
    return {"residual": h, "codes": slab.q.view(torch.float8_e4m3fn), "scales": slab.s.view(torch.float8_e8m0fnu)}


def run(state):
    if own:
        return _library(state)
    op = state["case"]["op"]
    return _plain_route(state) if op == "route" else _plain_experts(state) if op == "experts" else _plain_norm(state)


# ---------------------------------------------------------------------------
# The definition in 64 bits, from the representable values themselves.

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_pow2(e):
    return ((e + 1023) << 52).view(torch.float64)


def _exact_values(x, fmt):
    """float64 [rows, K] -> element values and exponents of its microscaled quantization."""
    g = x.view(x.shape[0], -1, GROUP)
    amax = g.abs().amax(dim=-1)
    # The exponent field of a float64 is floor(log2) + 1023.
    field = ((amax.view(torch.int64) >> 52) & 0x7FF) - 1023
    e = torch.where(amax > 0, field - (2 if fmt == "fp4" else 8), torch.full_like(field, -127)).clamp(-127, 127)
    v = g * _exact_pow2(-e)[..., None]
    a = v.abs()
    if fmt == "fp4":
        # Each midpoint between neighbours is crossed upwards strictly, or at
        # the midpoint itself where the upper neighbour has the even code.
        q = torch.zeros_like(a)
        for i in range(7):
            mid, step = 0.5 * (_E2M1[i] + _E2M1[i + 1]), _E2M1[i + 1] - _E2M1[i]
            q += step * ((a >= mid) if (i + 1) % 2 == 0 else (a > mid)).to(torch.float64)
    else:
        ex = (((a.view(torch.int64) >> 52) & 0x7FF) - 1023).clamp(min=-6)
        step = _exact_pow2(ex - 3)
        q = (torch.round(a / step) * step).clamp(max=448.0)
    return torch.copysign(q, v), e


def _exact_quantized(x, fmt):
    q, e = _exact_values(x, fmt)
    return (q * _exact_pow2(e)[..., None]).view(x.shape)


def _exact_weights(q, s, N, K):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float64, device=DEV)
    out = torch.empty((N, K), dtype=torch.float64, device=DEV)
    for k0 in range(0, K, 128):
        n = min(128, K - k0)
        b = torch.cat([q[k0 // 128, :, c].reshape(-1, 16) for c in range(n // 32)], dim=1)[:N].to(torch.int64)
        sc = _exact_pow2(s[k0 // 128, :N, : n // 32].to(torch.int64) - 127).repeat_interleave(GROUP, dim=1)
        out[:, k0 : k0 + n : 2] = table[b & 15]
        out[:, k0 + 1 : k0 + n : 2] = table[b >> 4]
        out[:, k0 : k0 + n] *= sc
    return out


def _exact_route(st):
    c = st["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = st["logits"].to(torch.float64)
    if c["scores"] == "softmax":
        s = torch.exp(l - torch.logsumexp(l, dim=1, keepdim=True))
    else:
        s = torch.sigmoid(l)
    key = l if st["bias"] is None else (s + st["bias"].to(torch.float64)).to(torch.float32).to(torch.float64)
    key = key.clone()
    index = torch.arange(E, device=l.device)
    if G > 1:
        v = key.view(T, G, -1)
        top2 = v.topk(min(2, E // G), dim=2).values
        score = top2.to(torch.float32).sum(dim=2) if st["bias"] is not None else top2[..., 0]
        left = score.to(torch.float64)
        kept = torch.zeros((T, G), dtype=torch.bool, device=l.device)
        for _ in range(c["top"]):
            at = (left == left.amax(dim=1, keepdim=True)).to(torch.int8).argmax(dim=1, keepdim=True)
            kept.scatter_(1, at, True)
            left = left.scatter(1, at, -math.inf)
        key[~kept[:, index // (E // G)]] = -math.inf
    ids = torch.empty((T, k), dtype=torch.int64, device=l.device)
    for j in range(k):
        m = key.amax(dim=1, keepdim=True)
        ids[:, j] = torch.where(key == m, index, E).amin(dim=1)
        key.scatter_(1, ids[:, j : j + 1], -math.inf)
    w = s.gather(1, ids)
    return {"ids": ids.to(torch.int32), "weights": 2.5 * w / w.sum(dim=1, keepdim=True)}


def _exact_experts(st):
    c = st["case"]
    H, I, act = c["H"], c["I"], c["act"]
    x = _exact_quantized(st["x"].to(torch.float64), act)
    y = torch.zeros((c["T"], H), dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        t, j = (st["ids"] == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        u = torch.mm(x[t], _exact_weights(st["up"][0][e], st["up"][1][e], 2 * I, H).t())
        a = (u[:, :I] * torch.sigmoid(u[:, :I]) * u[:, I:]).to(torch.float32).to(torch.bfloat16).to(torch.float64)
        o = torch.mm(_exact_quantized(a, act), _exact_weights(st["down"][0][e], st["down"][1][e], H, I).t())
        y.index_add_(0, t, o * st["weights"][t, j].to(torch.float64)[:, None])
    return y


def _exact_norm(st):
    c, M, K = st["case"], st["case"]["M"], st["case"]["K"]
    row = torch.arange(M, device=DEV)
    n = st["x"].to(torch.float64)
    if st["post"] is not None:
        n = n / torch.sqrt(torch.sum(n * n, dim=1) / K + EPS)[:, None] * st["post"].to(torch.float64)[None, :]
    if st["gate"] is not None:
        n *= st["gate"].to(torch.float64)[row * st["gate"].shape[0] // M]
    n += st["alpha"] * st["residual"].to(torch.float64)
    h = n.to(torch.float32).to(st["residual"].dtype).to(torch.float64)
    d = h - torch.sum(h, dim=1, keepdim=True) / K if c["kind"] == "layer" else h
    y = d / torch.sqrt(torch.sum(d * d, dim=1) / K + EPS)[:, None] * st["gain"].to(torch.float64)[None, :]
    if st["scale"] is not None:
        at = row * st["scale"].shape[0] // M
        y = y * (st["scale"].to(torch.float64)[at] + 1.0) + st["shift"].to(torch.float64)[at]
    y = y.to(torch.float32).to(torch.bfloat16).to(torch.float64)
    q, e = _exact_values(y, "fp8")
    R = _rows(M)
    codes = torch.zeros((K // 64, R, 64), dtype=torch.float64, device=DEV)
    codes[:, :M] = q.view(M, K // 64, 64).transpose(0, 1)
    scales = torch.full((K // 64, R, 2), 2.0**-127, dtype=torch.float64, device=DEV)
    scales[:, :M] = _exact_pow2(e).view(M, K // 64, 2).transpose(0, 1)
    return {"residual": h, "codes": codes, "scales": scales}


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "experts": _exact_experts, "norm": _exact_norm}[case["op"]](st)
