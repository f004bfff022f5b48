"""Cases of the 4-bit products: MXFP4 quantisation, the products of packed
MXFP4 and NVFP4 matrices, and a mixture-of-experts layer over NVFP4 experts.

Each case can be computed two ways: by the library's entry points (`own`
true) or in plain torch operations in float32 (`own` false).  `exact` gives
the same results from the definitions in float64.

Formats: an E2M1 nibble n has the value {0, .5, 1, 1.5, 2, 3, 4, 6}[n & 7],
negative with bit 3 set, two to a byte, the first in the low half.  MXFP4 has
an E8M0 byte e (scale 2^(e-127)) per 32 elements, NVFP4 an E4M3 byte per 16
and one float32 scale per tensor (per expert in the layer).
"""
import math

import torch

own = False

DEV = "cuda"
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)     # between neighbouring E2M1 magnitudes
MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# limits of the drawn cases: those of the largest listed ones
QUANT_ELEMS = 65536 * 4096
MM_WORK = 8192 * 12288 * 4096


# ---------------------------------------------------------------- the cases

def listed():
    mm = lambda op, name, t, o, k: {"name": name, "op": op, "tokens": t, "out": o, "k": k}
    moe = lambda name, t: {"name": name, "op": "moe", "tokens": t, "experts": 128, "top_k": 8, "hidden": 7168,
                           "inter": 2048}
    return [
        # the inputs of a Linear for a handful of sequences in decoding: a launch's latency
        {"name": "mxquant 3x4096", "op": "mxquant", "rows": 3, "k": 4096},
        # a calibration chunk's activations, out to MXFP4 and back: bandwidth
        {"name": "mxquant 65536x4096", "op": "mxquant", "rows": 65536, "k": 4096},
        # gate projection of the MLP set for one sequence: the weight is read once
        mm("mx", "mx gate t1", 1, 12288, 4096),
        # down projection for a short ragged batch: too few tiles for the card, K is split
        mm("mx", "mx down t333", 333, 4096, 12288),
        # gate projection over a prompt batch: matrix-core bound
        mm("mx", "mx gate t8192", 8192, 12288, 4096),
        # down projection for five sequences, activations left in bf16
        mm("w4a16", "w4a16 down t5", 5, 4096, 12288),
        # down projection over a prompt batch, activations left in bf16
        mm("w4a16", "w4a16 down t8192", 8192, 4096, 12288),
        # q projection of the 2048-wide decoder for sixteen sequences: the smallest product
        mm("w4a4", "w4a4 q_proj t16", 16, 2048, 2048),
        # gate projection over a ragged prompt batch, everything in 4 bits
        mm("w4a4", "w4a4 gate t4095", 4095, 12288, 4096),
        # the expert set of the cast (128 experts of 2048 x 7168) for one token,
        moe("moe t1", 1),
        # for a decoding batch,
        moe("moe t16", 16),
        # and for a batch that reaches nearly every expert
        moe("moe t61", 61),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mxquant", "mx", "w4a16", "w4a4", "moe"])
    if op == "mxquant":
        k = 32 * _logint(rng, 1, 384)
        return {"op": op, "rows": _logint(rng, 1, min(65536, QUANT_ELEMS // k)), "k": k}
    if op == "moe":
        experts = _logint(rng, 8, 128)
        return {"op": op, "tokens": _logint(rng, 1, 64), "experts": experts, "top_k": rng.randint(1, 8),
                "hidden": 16 * _logint(rng, 16, 448), "inter": 16 * _logint(rng, 8, 128)}
    unit = 32 if op == "mx" else 16
    while True:
        t, o, k = _logint(rng, 1, 8192), _logint(rng, 64, 12288), unit * _logint(rng, 256 // unit, 12288 // unit)
        if t * o * k <= MM_WORK:
            return {"op": op, "tokens": t, "out": o, "k": k}


def work(case):
    op = case["op"]
    if op == "mxquant":
        n = case["rows"] * case["k"]
        # quantise: 2 bytes in, 1/2 + 1/32 out; dequantise: the same backwards
        return {"bytes": 2 * (2 * n + n // 2 + n // 32), "flops": 2 * n}
    if op == "moe":
        t, e, kk, d, f = (case[c] for c in ("tokens", "experts", "top_k", "hidden", "inter"))
        # experts that at least one of t * top_k evenly spread choices reaches
        hit = e * (1.0 - (1.0 - kk / e) ** t)
        return {"bytes": int(hit * 3 * d * f * 9 / 16) + t * (4 * e + 4 * d + 8 * kk), "flops": 6 * t * kk * d * f}
    t, o, k = case["tokens"], case["out"], case["k"]
    per = 17 / 32 if op == "mx" else 9 / 16
    x = 2.0 if op == "w4a16" else per
    return {"bytes": int(t * k * x + o * k * per) + 2 * t * o, "flops": 2 * t * o * k}


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _acts(g, rows, k):
    """Laplace activations with a few outlier channels, bf16."""
    u = torch.rand((rows, k), generator=g, device=DEV) - 0.5
    x = torch.log1p(u.abs().mul_(-2.0).clamp_(min=-0.9999999)) * -torch.sign(u)
    x[:, torch.randint(0, k, (8,), generator=g, device=DEV)] *= 40.0
    return x.to(torch.bfloat16)


def _nibbles(q):
    """Packed E2M1 nibbles of scaled float32 values [rows, k]."""
    n = torch.bucketize(q.abs(), torch.tensor(MIDS, device=DEV)).to(torch.uint8)
    n |= (q < 0).to(torch.uint8) << 3
    return n[:, 0::2] | (n[:, 1::2] << 4)


def _mx_inputs(x):
    """Some MXFP4 form of x (any reasonable rounding: it is input data)."""
    b = x.float().view(x.shape[0], -1, 32)
    e = (torch.frexp(b.abs().amax(-1)).exponent - 3).clamp(-127, 127)
    q = torch.ldexp(b, -e[..., None]).view(x.shape)
    return _nibbles(q), (e + 127).to(torch.uint8)


def _nv_inputs(x):
    """Some NVFP4 form of x: nibbles, E4M3 codes and the tensor scale."""
    b = x.float().view(x.shape[0], -1, 16)
    am = b.abs().amax(-1)
    s2 = (am.amax() / 2688.0).clamp(min=1e-30)
    codes = (am / (6.0 * s2)).clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8).clamp(min=1)
    d = _e4m3(codes) * s2
    return _nibbles((b / d[..., None]).view(x.shape)), codes, s2.view(1)


def _e4m3(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _experts(g, e, mats, rows, k):
    """Packed experts as the MXFP4 -> NVFP4 cast leaves them: uniform nibbles,
    power-of-two block scales over a few binades with some ordinary E4M3 codes
    among them (requantised blocks), one tensor scale per expert that puts the
    products of unit inputs near 1."""
    p = torch.randint(0, 256, (e, mats, rows, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    c = torch.randint(5, 13, (e, mats, rows, k // 16), generator=g, device=DEV, dtype=torch.uint8) << 3
    odd = torch.rand((e, mats, rows, k // 16), generator=g, device=DEV) < 0.05
    c |= odd.to(torch.uint8) * 5
    s2 = torch.exp2(-torch.randint(4, 6, (e,), generator=g, device=DEV).float()) / math.sqrt(k)
    return p, c, s2


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"op": op}
    if op == "mxquant":
        st["x"] = _acts(g, case["rows"], case["k"])
    elif op == "moe":
        t, e, d, f = case["tokens"], case["experts"], case["hidden"], case["inter"]
        st["top_k"] = min(case["top_k"], e)
        st["x"] = torch.randn((t, d), generator=g, device=DEV).to(torch.bfloat16)
        st["logits"] = torch.randn((t, e), generator=g, device=DEV)
        st["w13"] = _experts(g, e, 2, f, d)
        st["w2"] = _experts(g, e, 1, d, f)
    else:
        t, o, k = case["tokens"], case["out"], case["k"]
        x = _acts(g, t, k)
        w = torch.randn((o, k), generator=g, device=DEV) * 0.02
        if op == "mx":
            st["x"], st["w"] = _mx_inputs(x), _mx_inputs(w)
        else:
            st["x"] = (x,) if op == "w4a16" else _nv_inputs(x)
            st["w"] = _nv_inputs(w)
    if own:
        import nvfp4_post_quantization_amd as nq
        nq.load()
        st["nq"] = nq
        if op == "moe":
            n = nq.moe_workspace_bytes(t, st["top_k"], case["inter"])
        elif op == "mx":
            n = nq.mxfp4_matmul_workspace_bytes(t, o, k)
        elif op != "mxquant":
            n = nq.matmul_workspace_bytes(t, o, k)
        else:
            n = 0
        st["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["op"]
    if own:
        nq = state["nq"]
        if op == "mxquant":
            return nq.mxfp4_dequant(*nq.mxfp4_quantize(state["x"]))
        if op == "mx":
            return nq.mxfp4_matmul(*state["x"], *state["w"], workspace=state["ws"])
        if op == "w4a16":
            return nq.matmul_w4a16(*state["x"], *state["w"], workspace=state["ws"])
        if op == "w4a4":
            return nq.matmul_w4a4(*state["x"], *state["w"], workspace=state["ws"])
        ids, wts = nq.moe_route(state["logits"], state["top_k"])
        y = nq.moe_forward(state["x"], ids, wts, *state["w13"], *state["w2"], workspace=state["ws"])
        return y, ids, wts
    if op == "mxquant":
        return _plain_mx_round_trip(state["x"])
    if op == "mx":
        return (_plain_mx(*state["x"]) @ _plain_mx(*state["w"]).t()).to(torch.bfloat16)
    if op == "w4a16":
        wp, wc, ws = state["w"]
        return ((state["x"][0].float() @ _plain_nv(wp, wc).t()) * ws).to(torch.bfloat16)
    if op == "w4a4":
        xp, xc, xs = state["x"]
        wp, wc, ws = state["w"]
        return ((_plain_nv(xp, xc) @ _plain_nv(wp, wc).t()) * ws * xs).to(torch.bfloat16)
    return _plain_moe(state)


def _pairs():
    """[256, 2] float32: the two E2M1 values of every byte."""
    b = torch.arange(256, device=DEV)
    m = torch.tensor(MAGS + tuple(-v for v in MAGS), device=DEV)
    return torch.stack((m[b & 15], m[b >> 4]), 1)


def _plain_mx(packed, e8m0):
    v = _pairs()[packed.int()].view(*e8m0.shape, 32)
    return torch.ldexp(v, (e8m0.int() - 127)[..., None]).view(*packed.shape[:-1], -1)


def _plain_nv(packed, codes):
    v = _pairs()[packed.int()].view(*codes.shape, 16)
    return (v * _e4m3(codes)[..., None]).view(*packed.shape[:-1], -1)


def _plain_mx_round_trip(x):
    b = x.float().view(x.shape[0], -1, 32)
    am = b.abs().amax(-1)
    e = torch.where(am > 0, torch.frexp(am).exponent - 3, -127).clamp(-127, 127)[..., None]
    q = torch.ldexp(b, -e)
    a = q.abs()
    idx = torch.zeros_like(b, dtype=torch.int32)
    for i, m in enumerate(MIDS):
        idx += (a >= m) if i % 2 else (a > m)         # ties go to the even index
    v = torch.tensor(MAGS, device=DEV)[idx]
    return torch.ldexp(torch.copysign(v, q), e).view(x.shape).to(torch.bfloat16)


def _plain_route(logits, top_k):
    v, i = torch.sort(logits, dim=1, descending=True, stable=True)
    v, i = v[:, :top_k], i[:, :top_k]
    p = torch.exp(v - v[:, :1])
    return i.int(), p / p.sum(1, keepdim=True)


def _plain_moe(state):
    x = state["x"].float()
    ids, wts = _plain_route(state["logits"], state["top_k"])
    (p13, c13, s13), (p2, c2, s2) = state["w13"], state["w2"]
    t, kk = ids.shape
    y = torch.zeros_like(x)
    if t * kk < p13.shape[0]:
        for s in range(kk):                           # few choices: fetch the experts chosen
            e = ids[:, s].long()
            w = _plain_nv(p13[e], c13[e]).flatten(1, 2)
            gu = torch.bmm(w, x[:, :, None]).view(t, 2, -1) * s13[e][:, None, None]
            h = gu[:, 0] / (1.0 + torch.exp(-gu[:, 0])) * gu[:, 1]
            w = _plain_nv(p2[e], c2[e])[:, 0]
            y += torch.bmm(w, h[:, :, None])[:, :, 0] * (s2[e] * wts[:, s])[:, None]
    else:
        for e in range(p13.shape[0]):                 # most experts are chosen: each in turn, all tokens
            gu = x @ _plain_nv(p13[e], c13[e]).flatten(0, 1).t() * s13[e]
            gate, up = gu.chunk(2, dim=1)
            h = gate / (1.0 + torch.exp(-gate)) * up
            share = (wts * (ids == e)).sum(1, keepdim=True) * s2[e]
            y += (h @ _plain_nv(p2[e, 0], c2[e, 0]).t()) * share
    return y.to(torch.bfloat16), ids, wts


# ---------------------------------------------------------------- float64

def _e2m1_64(packed):
    """float64 E2M1 values from the bits: exponent field e, mantissa bit m."""
    n = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    e, m = ((n >> 1) & 3).double(), (n & 1).double()
    v = torch.where(e == 0, 0.5 * m, torch.exp2(e - 1.0) * (1.0 + 0.5 * m))
    return torch.where(n >= 8, -v, v)


def _mx_64(packed, e8m0):
    return _e2m1_64(packed) * torch.exp2(e8m0.double() - 127.0).repeat_interleave(32, -1)


def _nv_64(packed, codes, s2):
    e, m = ((codes >> 3) & 15).double(), (codes & 7).double()
    c = torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e - 10.0) * (8.0 + m))
    return _e2m1_64(packed) * (c * s2.double()).repeat_interleave(16, -1)


def _quant_64(x):
    """Nearest E2M1 value (even index on ties) at the block's power of two."""
    x = x.double()
    b = x.view(x.shape[0], -1, 32)
    am = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(am > 0, am, 2.0 ** -125))) - 2.0
    # the logarithm may round up to the next whole number just below it
    e = torch.where(torch.exp2(e + 2.0) > am, torch.where(am > 0, e - 1.0, e), e).clamp(-127.0, 127.0)
    a = (b.abs() / torch.exp2(e)).clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    v = torch.round(a / step) * step                  # round half to even: steps of one binade
    return (torch.copysign(v, b) * torch.exp2(e)).view(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "mxquant":
        return torch.cat([_quant_64(x) for x in st["x"].split(8192)])
    if op == "moe":
        return _moe_64(st)
    if op == "mx":
        xs, ws = _mx_64(*st["x"]), _mx_64(*st["w"])
    else:
        xs = st["x"][0].double() if op == "w4a16" else _nv_64(*st["x"])
        ws = _nv_64(*st["w"])
    return torch.matmul(xs, ws.t())


def _moe_64(st):
    x = st["x"].double()
    z = st["logits"].double()
    kk = st["top_k"]
    y = torch.zeros_like(x)
    taken = torch.zeros_like(z, dtype=torch.bool)
    ids, val = [], []
    for _ in range(kk):                               # argmax takes the lowest index among equals here
        m = z.masked_fill(taken, -math.inf).amax(1, keepdim=True)
        i = torch.where((z == m) & ~taken, torch.arange(z.shape[1], device=DEV), z.shape[1]).amin(1, keepdim=True)
        taken.scatter_(1, i, True)
        ids.append(i)
        val.append(m)
    ids, wts = torch.cat(ids, 1), torch.softmax(torch.cat(val, 1), 1)
    (p13, c13, s13), (p2, c2, s2) = st["w13"], st["w2"]
    for e in torch.unique(ids).tolist():
        t, s = torch.nonzero(ids == e, as_tuple=True)
        gate = x[t] @ _nv_64(p13[e, 0], c13[e, 0], s13[e]).t()
        up = x[t] @ _nv_64(p13[e, 1], c13[e, 1], s13[e]).t()
        h = gate * torch.sigmoid(gate) * up
        y.index_add_(0, t, (h @ _nv_64(p2[e, 0], c2[e, 0], s2[e]).t()) * wts[t, s][:, None])
    return y, ids.int(), wts
