"""Cases of what stands around the packed products: tokens sorted by expert and
back with its gradient, the expert layer for many tokens, and low-rank adapters
of many requests beside a shared W4A16 projection.

Each case can be computed two ways: by the library's entry points (`own`
true) or in plain torch operations in float32 (`own` false).  `exact` gives
the same results from the definitions in float64.

A choice is a token and one of its top_k places, c = token * top_k + place.
Sorted rows are the choices whose id lies in 0 .. experts-1, by expert, then by
choice: order[row] = choice (-1 behind the last row), place[choice] = row (-1
for a choice without), offsets[e] = the first row of expert e.

Formats: an E2M1 nibble n has the value {0, .5, 1, 1.5, 2, 3, 4, 6}[n & 7],
negative with bit 3 set, two to a byte, the first in the low half; NVFP4 has
an E4M3 byte per 16 of them and a float32 scale per tensor (per expert).
"""
import math

import torch

own = False

DEV = "cuda"
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)     # between neighbouring E2M1 magnitudes
MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# limits of the drawn cases: those of the largest listed ones
SORT_MOST = 65536 * 8
MOVE_MOST = 8192 * 8 * 7168
LAYER_MOST = 8192 * 8 * 7168 * 2048
LORA_MOST = 8192 * 12288 * 4096


# ---------------------------------------------------------------- the cases

def listed():
    sort = lambda name, t, k, e: {"name": name, "op": "sort", "tokens": t, "top_k": k, "experts": e}
    rows = lambda op, name, t, k, e, d: {"name": name, "op": op, "tokens": t, "top_k": k, "experts": e, "hidden": d}
    layer = lambda name, t: {"name": name, "op": "layer", "tokens": t, "top_k": 8, "experts": 128, "hidden": 7168,
                             "inter": 2048}
    lora = lambda name, t, o, k, a, r: {"name": name, "op": "lora", "tokens": t, "out": o, "k": k, "adapters": a,
                                        "rank": r}
    return [
        # the choices of a decoding batch: a launch's latency
        sort("sort 61x8", 61, 8, 128),
        # those of a calibration chunk
        sort("sort 65536x8", 65536, 8, 128),
        # the tokens of a decoding batch to their experts and back
        rows("move", "move 61x8", 61, 8, 128, 7168),
        # a prompt batch: bandwidth
        rows("move", "move 8192x8", 8192, 8, 128, 7168),
        # the gradient of both ways for a ragged batch of the 2048-wide decoder
        rows("grad", "grad 333x4", 333, 4, 24, 2048),
        # and for a training batch
        rows("grad", "grad 8192x8", 8192, 8, 128, 7168),
        # the expert layer just past a decoding batch: every expert read for a few tokens each
        layer("layer t100", 100),
        # a ragged prompt batch
        layer("layer t1023", 1023),
        # a prompt batch: matrix-core bound
        layer("layer t8192", 8192),
        # one sequence with its adapter at the gate projection: latency beside reading the weight once
        lora("lora gate t1", 1, 12288, 4096, 16, 16),
        # a decoding batch of as many requests as adapters, at the down projection
        lora("lora down t16", 16, 4096, 12288, 16, 16),
        # prompts of several requests
        lora("lora gate t8192", 8192, 12288, 4096, 8, 64),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "move", "grad", "layer", "lora"])
    experts = _logint(rng, 8, 256)
    top_k = rng.randint(1, 8)
    if op == "sort":
        return {"op": op, "tokens": _logint(rng, 1, SORT_MOST // top_k), "top_k": top_k, "experts": experts}
    if op in ("move", "grad"):
        hidden = 8 * _logint(rng, 8, 896)
        most = min(65536, MOVE_MOST // (hidden * top_k))
        return {"op": op, "tokens": _logint(rng, 1, most), "top_k": top_k, "experts": experts, "hidden": hidden}
    while op == "layer":
        case = {"op": op, "tokens": _logint(rng, 65, 8192), "top_k": top_k, "experts": min(experts, 128),
                "hidden": 16 * _logint(rng, 16, 448), "inter": 16 * _logint(rng, 8, 128)}
        if case["tokens"] * top_k * case["hidden"] * case["inter"] <= LAYER_MOST:
            return case
    while True:
        case = {"op": op, "tokens": _logint(rng, 1, 8192), "out": _logint(rng, 64, 12288),
                "k": 16 * _logint(rng, 16, 768), "adapters": _logint(rng, 1, 64), "rank": 8 * _logint(rng, 1, 16)}
        if case["tokens"] * case["out"] * case["k"] <= LORA_MOST:
            return case


def work(case):
    op, t = case["op"], case["tokens"]
    if op == "lora":
        o, k, a, r = (case[c] for c in ("out", "k", "adapters", "rank"))
        hit = a * (1.0 - (1.0 - 1.0 / a) ** t)          # adapters that evenly spread tokens reach
        return {"bytes": int(o * k * 9 / 16 + hit * r * (o + k) * 2) + 2 * t * (k + o) + 4 * t,
                "flops": 2 * t * (o * k + r * (o + k))}
    n, e = t * case["top_k"], case["experts"]
    if op == "sort":
        return {"bytes": 12 * n + 4 * e, "flops": 2 * n}
    if op == "layer":
        d, f = case["hidden"], case["inter"]
        hit = e * (1.0 - (1.0 - case["top_k"] / e) ** t)
        return {"bytes": int(hit * 3 * d * f * 9 / 16) + 4 * t * d + 8 * n, "flops": 6 * n * d * f}
    d = case["hidden"]
    if op == "move":
        # sort; x to every row; every row back with its weight
        return {"bytes": 12 * n + 4 * e + 2 * d * (t + n) + 2 * d * (n + t) + 8 * n, "flops": 2 * n * d}
    # dy and ys in, dys and dweights out; dxs in, dx out
    return {"bytes": 2 * d * (t + 2 * n) + 12 * n + 2 * d * (n + t) + 4 * n, "flops": 4 * n * d}


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


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _routes(g, tokens, top_k, experts, away=0.0):
    """Ids and softmax weights of a router that likes some experts better, a
    share `away` of the choices with an expert that lives elsewhere."""
    z = torch.randn((tokens, experts), generator=g, device=DEV)
    z += 0.5 * torch.randn((1, experts), generator=g, device=DEV)
    v, i = torch.topk(z, min(top_k, experts), dim=1)
    w = torch.softmax(v, 1)
    if away:
        gone = torch.rand(i.shape, generator=g, device=DEV) < away
        i = torch.where(gone, -1, i)
    return i.int().contiguous(), w.contiguous()


def _nibbles(q):
    """Packed E2M1 nibbles of scaled float32 values [rows, k]."""
    n = torch.bucketize(q.abs(), torch.tensor(MIDS, device=DEV)).to(torch.uint8)
    n |= (q < 0).to(torch.uint8) << 3
    return n[:, 0::2] | (n[:, 1::2] << 4)


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
    op, t = case["op"], case["tokens"]
    st = {"op": op}
    if op == "lora":
        o, k, a, r = (case[c] for c in ("out", "k", "adapters", "rank"))
        st["x"] = _acts(g, t, k)
        st["w"] = _nv_inputs(torch.randn((o, k), generator=g, device=DEV) * 0.02)
        # runs of tokens of one request, some requests without an adapter
        runs = max(1, min(t, 2 * a))
        who = torch.randint(0, a, (runs,), generator=g, device=DEV)
        who = torch.where(torch.rand((runs,), generator=g, device=DEV) < 0.1, -1, who)
        st["ids"] = who[torch.arange(t, device=DEV) * runs // t].int()
        st["lora"] = ((torch.randn((a, r, k), generator=g, device=DEV) / math.sqrt(k)).to(torch.bfloat16),
                      (torch.randn((a, o, r), generator=g, device=DEV) * 0.02).to(torch.bfloat16),
                      0.5 + torch.rand((a,), generator=g, device=DEV))
    else:
        e, kk = case["experts"], min(case["top_k"], case["experts"])
        st["experts"] = e
        st["ids"], st["wts"] = _routes(g, t, kk, e, 0.0 if op == "layer" else 0.02)
        if op == "layer":
            d, f = case["hidden"], case["inter"]
            st["x"] = _normal(g, t, d)
            st["w13"] = _experts(g, e, 2, f, d)
            st["w2"] = _experts(g, e, 1, d, f)
        elif op != "sort":
            d, n = case["hidden"], t * kk
            st["ys"] = _normal(g, n, d)
            st["rows"] = torch.zeros((n, d), dtype=torch.bfloat16, device=DEV)     # rows behind the last stay zero
            if op == "move":
                st["x"] = _normal(g, t, d)
            else:
                st["dy"], st["dxs"] = _normal(g, t, d), _normal(g, n, d)
                st["place"] = _plain_sort(st["ids"], e)[1]
    if own:
        import nvfp4_post_quantization_amd as nq
        nq.load()
        st["nq"] = nq
        if op == "lora":
            n = nq.matmul_lora_workspace_bytes(t, o, k, r)
        elif op == "layer":
            n = nq.moe_sorted_workspace_bytes(t, kk, e, d, f)
        else:
            n = nq.moe_sort_workspace_bytes(t, kk, e)
        st["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["op"]
    if own:
        nq = state["nq"]
        if op == "sort":
            return nq.moe_sort(state["ids"], state["experts"], workspace=state["ws"])
        if op == "move":
            order, place, offsets = nq.moe_sort(state["ids"], state["experts"], workspace=state["ws"])
            xs = nq.moe_dispatch(state["x"], place, out=state["rows"])
            return order, place, offsets, xs, nq.moe_combine(state["ys"], place, state["wts"])
        if op == "grad":
            dwts = torch.empty_like(state["wts"])
            nq.moe_combine_grad(state["dy"], state["ys"], state["place"], state["wts"], out=(state["rows"], dwts))
            return state["rows"], dwts, nq.moe_dispatch_grad(state["dxs"], state["place"])
        if op == "layer":
            return nq.moe_forward_sorted(state["x"], state["ids"], state["wts"], *state["w13"], *state["w2"],
                                         workspace=state["ws"])
        return nq.matmul_w4a16_lora(state["x"], *state["w"], state["ids"], *state["lora"], workspace=state["ws"])
    if op == "sort":
        return _plain_sort(state["ids"], state["experts"])
    if op == "move":
        order, place, offsets = _plain_sort(state["ids"], state["experts"])
        xs = _plain_dispatch(state["x"], place)
        return order, place, offsets, xs, _plain_combine(state["ys"], place, state["wts"]).to(torch.bfloat16)
    if op == "grad":
        return _plain_grad(state)
    if op == "layer":
        return _plain_layer(state)
    return _plain_lora(state)


def _plain_sort(ids, experts):
    n = ids.numel()
    key = ids.flatten()
    key = torch.where((key >= 0) & (key < experts), key, experts)
    key, order = torch.sort(key, stable=True)
    row = torch.arange(n, device=DEV)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=DEV, dtype=torch.int32))
    place = torch.empty(n, dtype=torch.int32, device=DEV)
    place[order] = torch.where(key < experts, row, -1).int()
    order = torch.where(key < experts, order, -1).int()
    return order, place.view(ids.shape), offsets.int()


def _plain_dispatch(x, place):
    rows = place.numel()
    xs = torch.zeros((rows + 1, x.shape[1]), dtype=x.dtype, device=DEV)       # the last one takes what has no row
    at = torch.where(place < 0, rows, place).long()
    for s in range(place.shape[1]):
        xs[at[:, s]] = x
    xs[rows] = 0
    return xs[:rows]


def _plain_combine(ys, place, weights=None):
    y = torch.zeros((place.shape[0], ys.shape[1]), dtype=torch.float32, device=DEV)
    for s in range(place.shape[1]):
        p = place[:, s].long()
        v = ys[p.clamp(min=0)].float()
        if weights is not None:
            v *= weights[:, s, None]
        y += torch.where(p[:, None] >= 0, v, 0.0)
    return y


def _plain_grad(state):
    place, wts, dy, ys = state["place"], state["wts"], state["dy"].float(), state["ys"]
    rows = place.numel()
    dys = torch.zeros((rows + 1, ys.shape[1]), dtype=torch.bfloat16, device=DEV)
    dwts = torch.zeros_like(wts)
    at = torch.where(place < 0, rows, place).long()
    for s in range(place.shape[1]):
        dys[at[:, s]] = (dy * wts[:, s, None]).to(torch.bfloat16)
        dot = (dy * ys[at[:, s].clamp(max=rows - 1)].float()).sum(1)
        dwts[:, s] = torch.where(place[:, s] >= 0, dot, 0.0)
    return dys[:rows].index_fill_(0, _behind(place), 0.0), dwts, _plain_combine(state["dxs"], place).to(torch.bfloat16)


def _behind(place):
    """Rows that no choice goes to."""
    free = torch.ones(place.numel() + 1, dtype=torch.bool, device=DEV)
    free[place.flatten().long()] = False                  # -1: the extra one
    return torch.nonzero(free[:-1])[:, 0]


def _pairs():
    """[256, 2] float32: the two E2M1 values of every byte."""
    b = torch.arange(256, device=DEV)
    m = torch.tensor(MAGS + tuple(-v for v in MAGS), device=DEV)
    return torch.stack((m[b & 15], m[b >> 4]), 1)


def _plain_nv(packed, codes):
    v = _pairs()[packed.int()].view(*codes.shape, 16)
    return (v * _e4m3(codes)[..., None]).view(*packed.shape[:-1], -1)


def _plain_layer(state):
    ids, wts = state["ids"], state["wts"]
    (p13, c13, s13), (p2, c2, s2) = state["w13"], state["w2"]
    order, place, offsets = _plain_sort(ids, p13.shape[0])
    xs = _plain_dispatch(state["x"], place).float()
    ys = torch.zeros_like(xs)
    bounds = offsets.tolist()
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if a == b:
            continue
        gate, up = (xs[a:b] @ _plain_nv(p13[e], c13[e]).flatten(0, 1).t() * s13[e]).chunk(2, dim=1)
        h = gate / (1.0 + torch.exp(-gate)) * up
        ys[a:b] = h @ _plain_nv(p2[e, 0], c2[e, 0]).t() * s2[e]
    return _plain_combine(ys, place, wts).to(torch.bfloat16)


def _plain_lora(state):
    x, ids = state["x"].float(), state["ids"].long()
    wp, wc, ws = state["w"]
    a, b, scale = state["lora"]
    y = (x @ _plain_nv(wp, wc).t()) * ws
    if x.shape[0] < 2 * a.shape[0]:                       # few tokens: fetch the adapters chosen
        i = ids.clamp(min=0)
        u = torch.bmm(a[i].float(), x[:, :, None]) * scale[i, None, None]
        y += torch.where(ids[:, None] >= 0, torch.bmm(b[i].float(), u)[:, :, 0], 0.0)
    else:                                                 # else each in turn, all tokens
        for j in range(a.shape[0]):
            u = (x @ a[j].float().t()) * torch.where(ids == j, scale[j], 0.0)[:, None]
            y += u @ b[j].float().t()
    return y.to(torch.bfloat16)


# ---------------------------------------------------------------- float64

def _e2m1_64(packed):
    """float64 E2M1 values from the bits: exponent field e, mantissa bit m."""
    n = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    e, m = ((n >> 1) & 3).double(), (n & 1).double()
    v = torch.where(e == 0, 0.5 * m, torch.exp2(e - 1.0) * (1.0 + 0.5 * m))
    return torch.where(n >= 8, -v, v)


def _nv_64(packed, codes, s2):
    e, m = ((codes >> 3) & 15).double(), (codes & 7).double()
    c = torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e - 10.0) * (8.0 + m))
    return _e2m1_64(packed) * (c * s2.double()).repeat_interleave(16, -1)


def _sort_64(ids, experts):
    """By counting: a choice's row is the number of those before it."""
    flat = ids.flatten()
    place = torch.full_like(flat, -1)
    order = torch.full_like(flat, -1)
    offsets = [0]
    for e in range(experts):
        c = torch.nonzero(flat == e)[:, 0]
        r = torch.arange(offsets[-1], offsets[-1] + c.numel(), device=DEV)
        place[c] = r.int()
        order[r] = c.int()
        offsets.append(offsets[-1] + c.numel())
    return order, place.view(ids.shape), torch.tensor(offsets, dtype=torch.int32, device=DEV)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "lora":
        return _lora_64(st)
    if op == "layer":
        return _layer_64(st)
    order, place, offsets = _sort_64(st["ids"], st["experts"])
    if op == "sort":
        return order, place, offsets
    kk = place.shape[1]
    total = int(offsets[-1])
    choice = order[:total].long()
    token = choice // kk
    w = st["wts"].flatten().double()
    ys = st["ys"][:total].double()
    if op == "move":
        xs = torch.zeros_like(st["ys"])
        xs[:total] = st["x"][token]
        y = torch.zeros(st["x"].shape, dtype=torch.float64, device=DEV)
        y.index_add_(0, token, ys * w[choice, None])
        return order, place, offsets, xs, y
    dy = st["dy"].double()
    dys = torch.zeros(st["ys"].shape, dtype=torch.float64, device=DEV)
    dys[:total] = dy[token] * w[choice, None]
    dw = torch.zeros_like(w)
    dw[choice] = torch.cat([(dy[t] * v).sum(1) for t, v in zip(token.split(8192), ys.split(8192))])
    dx = torch.zeros(dy.shape, dtype=torch.float64, device=DEV)
    dx.index_add_(0, token, st["dxs"][:total].double())
    return dys, dw.view(place.shape), dx


def _layer_64(st):
    x, ids, wts = st["x"].double(), st["ids"], st["wts"].double()
    (p13, c13, s13), (p2, c2, s2) = st["w13"], st["w2"]
    y = torch.zeros_like(x)
    for e in torch.unique(ids).tolist():
        t, s = torch.nonzero(ids == e, as_tuple=True)
        gate = x[t] @ _nv_64(p13[e, 0], c13[e, 0], s13[e]).t()
        up = x[t] @ _nv_64(p13[e, 1], c13[e, 1], s13[e]).t()
        h = gate * torch.sigmoid(gate) * up
        y.index_add_(0, t, (h @ _nv_64(p2[e, 0], c2[e, 0], s2[e]).t()) * wts[t, s][:, None])
    return y


def _lora_64(st):
    x, ids = st["x"].double(), st["ids"]
    a, b, scale = st["lora"]
    y = x @ _nv_64(*st["w"]).t()
    for j in torch.unique(ids).tolist():
        if j >= 0:
            t = torch.nonzero(ids == j)[:, 0]
            y[t] += (x[t] @ a[j].double().t()) @ b[j].double().t() * scale[j].double()
    return y
