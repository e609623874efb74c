"""Measured cases of the mixture-of-experts layers for a few tokens and of the linear layer on 8-bit codes.

Operators (``op`` in a case):
  moe_bf16, moe_int8, moe_int4
         routing, gate, up, activation, down and the weighted sum over a token's experts, on bf16
         weights, on 8-bit codes (tokens and h quantised per token) and on 4-bit group-scaled codes
  int8   y = (codes of x)(codes of W)^T times the scales of token and channel, both given
  w8a8   x quantised to codes and scales per token, then the same product

``own`` chooses between the plain forms below (32-bit torch arithmetic) and the library's entry
points.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------- cases
def _moe(op, M, E, topk, H, I, **more):
    c = dict(op=op, M=M, E=E, topk=topk, H=H, I=I, limit=0.0, renorm=False)
    if op == "moe_int4":
        c.update(group=128, zeros=False, scale="bf16")
    c.update(more)
    return c


def listed():
    return [
        # one token through a small layer: the latency of a call
        dict(_moe("moe_int4", 1, 8, 2, 1024, 512), name="moe_int4 1 of 8 512x1024"),
        # one token decoding through a large layer, 8 of 256 experts
        dict(_moe("moe_int4", 1, 256, 8, 4096, 2048), name="moe_int4 1 of 256 2048x4096"),
        # an odd decode batch on a layer of mid-sized ragged experts, fine groups, asymmetric
        dict(_moe("moe_int4", 13, 60, 4, 2080, 1376, group=32, zeros=True, scale="fp16", renorm=True),
             name="moe_int4 13 of 60 1376x2080"),
        # the large layer on 8-bit codes, one token
        dict(_moe("moe_int8", 1, 256, 8, 4096, 2048), name="moe_int8 1 of 256 2048x4096"),
        # a decode batch that touches about 100 experts
        dict(_moe("moe_int8", 16, 256, 8, 4096, 2048, limit=10.0), name="moe_int8 16 of 256 2048x4096"),
        # the unquantised large layer, one token
        dict(_moe("moe_bf16", 1, 256, 8, 4096, 2048), name="moe_bf16 1 of 256 2048x4096"),
        # few experts, several tokens each, ragged sizes
        dict(_moe("moe_bf16", 7, 16, 2, 2056, 1032, limit=10.0, renorm=True), name="moe_bf16 7 of 16 1032x2056"),
        # one token through gate and up of a 27B-class MLP, codes shared with other projections
        dict(op="int8", M=1, N=17408, K=5120, out="bf16", name="int8 1x17408x5120"),
        # an odd decode batch through the down projection
        dict(op="int8", M=19, N=5120, K=17408, out="bf16", name="int8 19x5120x17408"),
        # a prompt of an odd length, sums kept in 32 bits for what follows
        dict(op="w8a8", M=777, N=10240, K=5120, out="fp32", name="w8a8 777x10240x5120"),
        # a long prompt through gate and up
        dict(op="w8a8", M=4096, N=17408, K=5120, out="bf16", name="w8a8 4096x17408x5120"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_WEIGHT_BYTES = {"moe_bf16": 2.0, "moe_int8": 1.0, "moe_int4": 0.5}


def draw(rng):
    op = rng.choice(["moe_bf16", "moe_int8", "moe_int4", "moe_int4", "int8", "w8a8"])
    if op in _WEIGHT_BYTES:
        M, E, I, H = _log(rng, 1, 64), _log(rng, 4, 256), 32 * _log(rng, 2, 64), 32 * _log(rng, 4, 128)
        topk = min(E, rng.choice([1, 2, 4, 6, 8]))
        # never more weights than the largest listed layer touches
        while min(E, M * topk) * 3 * I * H * _WEIGHT_BYTES[op] > 2.4e9:
            M = max(1, M // 2)
        c = _moe(op, M, E, topk, H, I, limit=rng.choice([0.0, 1.5, 10.0]), renorm=rng.random() < 0.5)
        if op == "moe_int4":
            c.update(group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5, scale=rng.choice(["bf16", "fp16"]))
        return c
    M = _log(rng, 1, 48) if op == "int8" else _log(rng, 1, 4096)
    return dict(op=op, M=M, N=_log(rng, 64, 17408), K=16 * _log(rng, 8, 320 if M > 48 else 1088),
                out=rng.choice(["bf16", "fp16", "fp32"]))


# --------------------------------------------------------------------------------------- inputs
def _activations(m, k, g):
    """Normal activations with a few channels several times larger, as normed hidden states have."""
    x = torch.randn(m, k, device="cuda", generator=g)
    gain = torch.where(torch.rand(k, device="cuda", generator=g) < 0.01, 6.0, 1.0)
    return (x * gain).to(torch.bfloat16)


def _codes(shape, g):
    return torch.randint(-127, 128, shape, device="cuda", generator=g, dtype=torch.int8)


def _channel_scales(shape, k, g):
    """Scales that give a sum over k codes of normal activations a size of about one."""
    return (torch.rand(shape, device="cuda", generator=g) + 0.5) / (73.0 * math.sqrt(k))


def _matrix(op, experts, n, k, case, g):
    """The weights of one projection of every expert: [E, n, k] as the format stores it."""
    if op == "moe_bf16":
        w = torch.randn(experts, n, k, device="cuda", generator=g, dtype=torch.bfloat16)
        return dict(w=w.mul_(1.0 / math.sqrt(k)))
    if op == "moe_int8":
        return dict(w=_codes((experts, n, k), g), s=_channel_scales((experts, n), k, g))
    groups = -(-k // case["group"])
    w = torch.randint(0, 256, (experts, n, k // 2), device="cuda", generator=g, dtype=torch.uint8)
    s = (torch.rand(experts, n, groups, device="cuda", generator=g) * 0.9 + 0.1) * (0.4 / math.sqrt(k))
    z = None
    if case["zeros"]:
        z = torch.randint(5, 12, (experts, n, groups), device="cuda", generator=g, dtype=torch.uint8)
    return dict(w=w, s=s.to(_DTYPES[case["scale"]]), z=z)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case=case)
    if case["op"] in _WEIGHT_BYTES:
        st["x"] = _activations(case["M"], case["H"], g)
        st["logits"] = torch.randn(case["M"], case["E"], device="cuda", generator=g).to(torch.bfloat16)
        st["w13"] = _matrix(case["op"], case["E"], 2 * case["I"], case["H"], case, g)
        st["w2"] = _matrix(case["op"], case["E"], case["H"], case["I"], case, g)
        return st
    x = _activations(case["M"], case["K"], g)
    st["w"] = _codes((case["N"], case["K"]), g)
    st["s"] = _channel_scales((case["N"],), case["K"], g)
    if case["op"] == "int8":
        st["xq"], st["xs"] = _quantised(x.float())
    else:
        st["x"] = x
    return st


# ---------------------------------------------------------------------------------- plain forms
def _quantised(x):
    """Codes and scale of every row: scale = max|x| / 127, code = x / scale rounded half to even."""
    s = x.abs().amax(dim=-1, keepdim=True)
    s = s / torch.full_like(s, 127.0)
    q = torch.where(s > 0, torch.round(x / s), torch.zeros_like(x)).clamp(-127, 127)
    return q.to(torch.int8), s.squeeze(-1)


def _routed(logits, topk, renorm):
    """Expert ids and weights of every token: the largest logits, equal ones to the lowest id."""
    e = torch.exp(logits.float() - logits.float().amax(dim=1, keepdim=True))
    p = e / e.sum(dim=1, keepdim=True)
    ids = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :topk]
    w = p.gather(1, ids)
    return ids, w / w.sum(dim=1, keepdim=True) if renorm else w


def _values(m, case, which=None):
    """A projection's weights in 32 bits, of the experts `which` or of all (8-bit: without scales)."""
    w = m["w"] if which is None else m["w"][which]
    if case["op"] != "moe_int4":
        return w.float()
    s = (m["s"] if which is None else m["s"][which]).float()
    q = torch.stack((w & 15, w >> 4), dim=-1).flatten(-2).float()
    at = torch.arange(q.shape[-1], device=q.device) // case["group"]
    if m["z"] is None:
        return (q - 8.0) * s[..., at]
    return (q - (m["z"] if which is None else m["z"][which]).float()[..., at]) * s[..., at]


def _product(x, m, case, which=None):
    """x [slots, tokens, k] times every slot's expert; an 8-bit layer quantises x's rows first."""
    w = _values(m, case, which).transpose(1, 2)
    if case["op"] != "moe_int8":
        return x @ w
    q, s = _quantised(x)
    return (q.float() @ w) * s.unsqueeze(-1) * (m["s"] if which is None else m["s"][which]).unsqueeze(1)


def _gated(g, u, limit):
    if limit:
        g, u = torch.clamp(g, max=limit), torch.clamp(u, min=-limit, max=limit)
    return g / (1.0 + torch.exp(-g)) * u


def _plain_moe(st):
    c = st["case"]
    m, k, i = c["M"], c["topk"], c["I"]
    ids, weights = _routed(st["logits"], k, c["renorm"])
    x = st["x"].float()
    if m * k < c["E"]:  # every (token, expert) pair with its expert's weights
        which = ids.reshape(-1)
        x = x.repeat_interleave(k, dim=0).unsqueeze(1)
    else:  # every token through every expert, those that it did not choose with weight zero
        which = None
        x = x.unsqueeze(0).expand(c["E"], -1, -1)
    gu = _product(x, st["w13"], c, which)
    h = _gated(gu[..., :i], gu[..., i:], c["limit"]).to(torch.bfloat16).float()
    o = _product(h, st["w2"], c, which)
    if which is not None:
        return (o.reshape(m, k, -1) * weights.unsqueeze(2)).sum(dim=1).to(torch.bfloat16)
    full = torch.zeros(m, c["E"], device=x.device).scatter_(1, ids, weights)
    return (o * full.t().unsqueeze(2)).sum(dim=0).to(torch.bfloat16)


def _run_plain(st):
    c = st["case"]
    if c["op"] in _WEIGHT_BYTES:
        return _plain_moe(st)
    xq, xs = (st["xq"], st["xs"]) if c["op"] == "int8" else _quantised(st["x"].float())
    y = (xq.float() @ st["w"].float().t()) * xs.unsqueeze(1) * st["s"]
    y = y.to(_DTYPES[c["out"]])
    return y if c["op"] == "int8" else dict(codes=xq, scale=xs, y=y)


def _run_own(st):
    import skinny_gemm_dequant_gb300 as ql
    c = st["case"]
    if c["op"] in _WEIGHT_BYTES:
        a, b = st["w13"], st["w2"]
        how = dict(router_logits=st["logits"], topk=c["topk"], renormalize=c["renorm"], swiglu_limit=c["limit"] or None)
        if c["op"] == "moe_bf16":
            return ql.moe_bf16(st["x"], a["w"], b["w"], **how)
        if c["op"] == "moe_int8":
            return ql.moe_int8(st["x"], a["w"], a["s"], b["w"], b["s"], **how)
        return ql.moe_int4(st["x"], a["w"], a["s"], b["w"], b["s"], a["z"], b["z"], group=c["group"], **how)
    if c["op"] == "int8":
        return ql.qlinear_int8(st["xq"], st["xs"], st["w"], st["s"], out_dtype=_DTYPES[c["out"]])
    xq, xs = ql.quantize_int8(st["x"])
    return dict(codes=xq, scale=xs, y=ql.qlinear_int8(xq, xs, st["w"], st["s"], out_dtype=_DTYPES[c["out"]]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------------------- work
def work(case):
    m = case["M"]
    if case["op"] in _WEIGHT_BYTES:
        e, k, i, h = case["E"], case["topk"], case["I"], case["H"]
        touched = e * (1.0 - (1.0 - k / e) ** m)  # experts that m tokens choose on average
        per = 3 * i * h * _WEIGHT_BYTES[case["op"]]
        if case["op"] == "moe_int8":
            per += 4 * (2 * i + h)
        elif case["op"] == "moe_int4":
            groups = 2 * i * -(-h // case["group"]) + h * -(-i // case["group"])
            per += groups * (3 if case["zeros"] else 2)
        return {"bytes": int(touched * per) + 4 * m * h + 2 * m * e, "flops": 6 * m * k * i * h}
    n, k = case["N"], case["K"]
    size = 4 if case["out"] == "fp32" else 2
    once = n * k + 4 * n + m * k + 4 * m + size * m * n
    return {"bytes": once + (2 * m * k if case["op"] == "w8a8" else 0), "flops": 2 * m * n * k}


# ------------------------------------------------------------------------- 64-bit definition
def _exact_weights(m, e, case):
    """The weights of expert e in 64 bits, scales included."""
    w = m["w"][e]
    if case["op"] == "moe_bf16":
        return w.double()
    if case["op"] == "moe_int8":
        return w.double() * m["s"][e].double()[:, None]
    codes = w.to(torch.int64)
    out = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.float64, device=w.device)
    out[:, 0::2] = (codes % 16).double()
    out[:, 1::2] = (codes // 16).double()
    for j in range(m["s"].shape[2]):
        part = out[:, j * case["group"]:(j + 1) * case["group"]]
        part -= 8.0 if m["z"] is None else m["z"][e, :, j:j + 1].double()
        part *= m["s"][e, :, j:j + 1].double()
    return out


def _exact_codes(v):
    """Whole codes and unit of every row.  The definition rounds the unit and the quotient to 32 bits:
    values of few bits fall on ties, which no other precision breaks alike."""
    top = v.abs().max(dim=1, keepdim=True).values
    unit = (top / 127.0).float().double()
    q = torch.round((v / unit.masked_fill(unit == 0, 1.0)).float().double())
    return q, unit


def _exact_moe(st):
    c = st["case"]
    x, logits = st["x"].double(), st["logits"].double()
    p = torch.softmax(logits, dim=1)
    chosen = torch.zeros_like(p)
    left = logits.clone()
    for _ in range(c["topk"]):
        best = (left == left.max(dim=1, keepdim=True).values).to(torch.int8).argmax(dim=1)
        rows = torch.arange(c["M"], device=x.device)
        chosen[rows, best] = p[rows, best]
        left[rows, best] = -math.inf
    if c["renorm"]:
        chosen /= chosen.sum(dim=1, keepdim=True)
    if c["op"] == "moe_int8":
        q, unit = _exact_codes(x)
        x = q * unit
    lim = c["limit"] or math.inf
    y = torch.zeros(c["M"], c["H"], dtype=torch.float64, device=x.device)
    for e in (chosen > 0).any(dim=0).nonzero().flatten().tolist():
        tok = (chosen[:, e] > 0).nonzero().flatten()
        w = _exact_weights(st["w13"], e, c)
        g, u = (x[tok] @ w.T).split(c["I"], dim=1)
        g = g.clamp(max=lim)
        h = g * torch.sigmoid(g) * u.clamp(-lim, lim)
        if c["op"] == "moe_int8":  # defined on h as it is kept, in 16 bits
            q, unit = _exact_codes(h.to(torch.bfloat16).double())
            h = q * unit
        y[tok] += chosen[tok, e, None] * (h @ _exact_weights(st["w2"], e, c).T)
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in _WEIGHT_BYTES:
        return _exact_moe(st)
    w = st["w"].double().T
    if case["op"] == "int8":
        return st["xs"].double()[:, None] * (st["xq"].double() @ w) * st["s"].double()
    q, s = _exact_codes(st["x"].double())
    return dict(codes=None, scale=s[:, 0], y=s * (q @ w) * st["s"].double())
