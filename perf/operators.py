"""Measured cases of the 4-bit linear layer and the gated feed-forward block.

Operators (``op`` in a case):
  int4        y = x W^T on 4-bit integer weights with group scales (and zero points)
  gated_int4  h = silu(a min(g, L)) clamp(u, -L, L) with g, u = x W13^T on such weights
  ffn         the same gated block on bf16 weights, forward only
  step        the gated block's forward with a checkpoint of g and u, then its backward pass

``own`` chooses between the plain forms below (32-bit torch arithmetic) and the library's entry
points.
"""
import math

import torch

own = False

CKPT_GROUP = 128  # columns of one 8-bit checkpoint scale


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token through a small projection: the latency of a call
        dict(name="int4 1x512x1024", op="int4", M=1, N=512, K=1024, group=128, zeros=False, scale="bf16"),
        # one token through the down projection of a 27B-class MLP, asymmetric weights
        dict(name="int4 1x5120x17408", op="int4", M=1, N=5120, K=17408, group=128, zeros=True, scale="bf16"),
        # a small decode batch through an attention-sized projection, fine groups
        dict(name="int4 16x10240x5120", op="int4", M=16, N=10240, K=5120, group=32, zeros=False, scale="fp16"),
        # one token through gate, up and the activation of the 27B-class MLP
        dict(name="gated_int4 1x17408x5120", op="gated_int4", M=1, I=17408, H=5120, group=128, zeros=True,
             scale="bf16", limit=0.0),
        # an odd decode batch through a narrow expert-sized block
        dict(name="gated_int4 7x2048x4096", op="gated_int4", M=7, I=2048, H=4096, group=64, zeros=False,
             scale="bf16", limit=10.0),
        # the unquantised block for one token
        dict(name="ffn 1x17408x5120", op="ffn", M=1, I=17408, H=5120, limit=0.0),
        # a decode batch of an odd size, ragged columns
        dict(name="ffn 13x2056x4096", op="ffn", M=13, I=2056, H=4096, limit=10.0),
        # a prompt of an odd length through the whole block
        dict(name="ffn 1000x17408x5120", op="ffn", M=1000, I=17408, H=5120, limit=0.0),
        # a short fine-tuning batch on a small ragged block
        dict(name="step 333x2040x1024", op="step", M=333, I=2040, H=1024, limit=0.0, save="int8"),
        # an ordinary batch on an expert-sized block, checkpoint kept in 16 bits
        dict(name="step 2048x2048x4096 bf16", op="step", M=2048, I=2048, H=4096, limit=10.0, save="bf16"),
        # a long batch on the whole block, checkpoint kept in 8 bits
        dict(name="step 4096x17408x5120", op="step", M=4096, I=17408, H=5120, limit=0.0, save="int8"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["int4", "gated_int4", "ffn", "step"])
    if op in ("int4", "gated_int4"):
        c = dict(op=op, M=_log(rng, 1, 32), group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5,
                 scale=rng.choice(["bf16", "fp16"]))
        if op == "int4":
            c.update(N=_log(rng, 64, 17408), K=32 * _log(rng, 8, 544))
        else:
            c.update(I=_log(rng, 64, 17408), H=32 * _log(rng, 8, 160), limit=rng.choice([0.0, 1.5, 10.0]))
        return c
    c = dict(op=op, M=_log(rng, 1, 4096), I=8 * _log(rng, 8, 2176), H=8 * _log(rng, 8, 640),
             limit=rng.choice([0.0, 1.5, 10.0]))
    if op == "step":
        c["save"] = rng.choice(["int8", "bf16"])
    return c


# --------------------------------------------------------------------------------------- inputs
def _activations(m, k, g):
    """Normal activations with a few channels several times larger, as normed hidden states have."""
    x = torch.randn(m, k, device="cuda", generator=g)
    gain = torch.where(torch.rand(k, device="cuda", generator=g) < 0.01, 6.0, 1.0)
    return (x * gain).to(torch.bfloat16)


def _int4_weights(n, k, case, g):
    groups = -(-k // case["group"])
    w = torch.randint(0, 256, (n, k // 2), device="cuda", generator=g, dtype=torch.uint8)
    s = (torch.rand(n, groups, device="cuda", generator=g) * 0.9 + 0.1) * (0.4 / math.sqrt(k))
    s = s.to(torch.bfloat16 if case["scale"] == "bf16" else torch.float16)
    z = None
    if case["zeros"]:
        z = torch.randint(5, 12, (n, groups), device="cuda", generator=g, dtype=torch.uint8)
    return w, s, z


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "int4":
        st["x"] = _activations(case["M"], case["K"], g)
        st["w"], st["s"], st["z"] = _int4_weights(case["N"], case["K"], case, g)
        return st
    m, i, h = case["M"], case["I"], case["H"]
    st["x"] = _activations(m, h, g)
    if case["op"] == "gated_int4":
        st["w"], st["s"], st["z"] = _int4_weights(2 * i, h, case, g)
        return st
    w = torch.randn(2 * i, h, device="cuda", generator=g)
    st["w"] = (w / math.sqrt(h)).to(torch.bfloat16)
    if case["op"] == "step":
        st["dh"] = (torch.randn(m, i, device="cuda", generator=g) * 0.02).to(torch.bfloat16)
    return st


# ---------------------------------------------------------------------------------- plain forms
def _dequantised(w, s, z, k, group):
    q = torch.stack((w & 15, w >> 4), dim=2).reshape(w.shape[0], k).float()
    zero = torch.full_like(s, 8, dtype=torch.float32) if z is None else z.float()
    at = torch.arange(k, device=w.device) // group
    return (q - zero[:, at]) * s.float()[:, at]


def _silu(t):
    return t / (1.0 + torch.exp(-t))


def _gated(g, u, limit):
    if limit:
        g, u = torch.clamp(g, max=limit), torch.clamp(u, min=-limit, max=limit)
    return _silu(g) * u


def _kept(v, save):
    """What the backward pass sees of g or u: its 8-bit codes times their scales, or bf16."""
    if save == "bf16":
        return v.to(torch.bfloat16).float()
    m, i = v.shape
    pad = -i % CKPT_GROUP
    t = torch.cat((v, v.new_zeros(m, pad)), dim=1).reshape(m, -1, CKPT_GROUP)
    s = t.abs().amax(dim=2, keepdim=True) / 127.0
    q = torch.where(s > 0, torch.round(t / s), torch.zeros_like(t)).clamp(-127, 127)
    return (q * s).reshape(m, -1)[:, :i]


def _backward(dh, x, w, g, u, limit):
    i = g.shape[1]
    gc, uc = g, u
    if limit:
        gc, uc = torch.clamp(g, max=limit), torch.clamp(u, min=-limit, max=limit)
    sig = 1.0 / (1.0 + torch.exp(-gc))
    du = dh * gc * sig
    dg = dh * uc * sig * (1.0 + gc * (1.0 - sig))
    if limit:
        du = du * (u.abs() <= limit)
        dg = dg * (g <= limit)
    dgu = torch.cat((dg, du), dim=1)
    return dgu @ w, dgu.t() @ x


def _run_plain(st):
    c = st["case"]
    x = st["x"].float()
    if c["op"] == "int4":
        return (x @ _dequantised(st["w"], st["s"], st["z"], c["K"], c["group"]).t()).to(torch.bfloat16)
    i = c["I"]
    if c["op"] == "gated_int4":
        w = _dequantised(st["w"], st["s"], st["z"], c["H"], c["group"])
    else:
        w = st["w"].float()
    gu = x @ w.t()
    g, u = gu[:, :i], gu[:, i:]
    h = _gated(g, u, c["limit"]).to(torch.bfloat16)
    if c["op"] != "step":
        return h
    dx, dw = _backward(st["dh"].float(), x, w, _kept(g, c["save"]), _kept(u, c["save"]), c["limit"])
    return dict(h=h, dx=dx.to(torch.bfloat16), dw=dw.to(torch.bfloat16))


def _run_own(st):
    import skinny_gemm_dequant_gb300 as ql
    c = st["case"]
    if c["op"] == "int4":
        return ql.qlinear_int4(st["x"], st["w"], st["s"], st["z"], group=c["group"])
    limit = c["limit"] or None
    if c["op"] == "gated_int4":
        return ql.gated_ffn_int4(st["x"], st["w"], st["s"], st["z"], group=c["group"], swiglu_limit=limit)
    if c["op"] == "ffn":
        return ql.gated_ffn(st["x"], st["w"], swiglu_limit=limit)
    h, saved = ql.gated_ffn(st["x"], st["w"], swiglu_limit=limit, save=c["save"])
    dx, dw = ql.gated_ffn_backward(st["dh"], st["x"], st["w"], saved, swiglu_limit=limit)
    return dict(h=h, dx=dx, dw=dw)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------------------- work
def work(case):
    m = case["M"]
    if case["op"] in ("int4", "gated_int4"):
        n, k = (case["N"], case["K"]) if case["op"] == "int4" else (2 * case["I"], case["H"])
        out = n if case["op"] == "int4" else n // 2
        per_group = 3 if case["zeros"] else 2
        return {"bytes": n * k // 2 + per_group * n * -(-k // case["group"]) + 2 * m * k + 2 * m * out,
                "flops": 2 * m * n * k}
    i, h = case["I"], case["H"]
    once = 4 * i * h + 2 * m * h + 2 * m * i  # W13, x and h
    if case["op"] == "ffn":
        return {"bytes": once, "flops": 4 * m * h * i}
    return {"bytes": once + 2 * m * i + 2 * m * h + 4 * i * h, "flops": 12 * m * h * i}


# ------------------------------------------------------------------------- 64-bit definition
def _exact_weights(st, rows, cols, group):
    codes = st["w"].to(torch.int64)
    w = torch.empty(rows, cols, dtype=torch.float64, device=codes.device)
    w[:, 0::2] = (codes % 16).double()
    w[:, 1::2] = (codes // 16).double()
    for j in range(st["s"].shape[1]):
        part = w[:, j * group:(j + 1) * group]
        part -= 8.0 if st["z"] is None else st["z"][:, j:j + 1].double()
        part *= st["s"][:, j:j + 1].double()
    return w


def _exact_kept(v, save):
    if save == "bf16":
        return v.to(torch.bfloat16).double()
    out = torch.zeros_like(v)
    for j in range(0, v.shape[1], CKPT_GROUP):
        part = v[:, j:j + CKPT_GROUP]
        top = part.abs().max(dim=1, keepdim=True).values
        unit = torch.where(top > 0, top / 127.0, torch.ones_like(top))
        out[:, j:j + CKPT_GROUP] = torch.round(part / unit) * unit
    return out


def exact(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    st = prepare(case, seed)
    x = st["x"].double()
    if case["op"] == "int4":
        return x @ _exact_weights(st, case["N"], case["K"], case["group"]).T
    i, lim = case["I"], case["limit"] or math.inf
    w = _exact_weights(st, 2 * i, case["H"], case["group"]) if case["op"] == "gated_int4" else st["w"].double()
    wg, wu = w[:i], w[i:]
    g, u = x @ wg.T, x @ wu.T
    gl = torch.minimum(g, torch.full_like(g, lim))
    h = gl * torch.sigmoid(gl) * u.clamp(-lim, lim)
    if case["op"] != "step":
        return h
    g, u = _exact_kept(g, case["save"]), _exact_kept(u, case["save"])
    gl = g.clamp(max=lim)
    sg = torch.sigmoid(gl)
    dh = st["dh"].double()
    dg = torch.where(g <= lim, dh * u.clamp(-lim, lim) * (sg + gl * sg * (1 - sg)), 0.0)
    du = torch.where(u.abs() <= lim, dh * gl * sg, 0.0)
    return dict(h=h, dx=dg @ wg + du @ wu, dw=torch.cat((dg.T @ x, du.T @ x)))
