"""Workloads of the feed-forward operators around the BitLinear layer.

Each case is one call (or one pair of gradient calls) of an operator on data
that lives on the GPU:

  act           y = f(x W^T + bias) + residual, the layer with its epilogue
  act_grad      dz = dy f'(z) and the bias gradient, the epilogue's backward
  grouped       the layer over rows sorted by expert, ragged sizes
  grouped_grad  dX and dW of the grouped layer
  adamw         one AdamW step over many tensors, states in 32 or 8 bits

`own` selects between the plain form (elementary torch operations in 32 bits)
and the library's calls.
"""

import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
BLOCK = 256                      # elements that share a scale in the 8-bit states
HASH_A, HASH_B = 0x9E3779B1, 0xB7E15163
SEED = 20240229                  # of the 8-bit states' rounding
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.95, 1e-5, 0.1


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _act(name, t, k, n_out, n, m, act, bias=True, residual=False, save_z=False):
    return dict(name=name, op="act", t=t, k=k, n_out=n_out, n=n, m=m, act=act, bias=bias, residual=residual,
                save_z=save_z)


def _grouped(name, rows, experts, idle, k, n_out, n, m, act="none", bias=False, op="grouped"):
    return dict(name=name, op=op, rows=rows, experts=experts, idle=idle, k=k, n_out=n_out, n=n, m=m, act=act,
                bias=bias)


def listed():
    return [
        # one token through an up-projection with squared ReLU
        _act("act_decode_t1", 1, 2560, 6912, 6, 8, "relu2"),
        # a training forward of a small model's up-projection, z kept for the backward
        _act("act_train_t2048", 2048, 896, 4864, 6, 8, "gelu", save_z=True),
        # a prefill's down-projection that adds the residual stream
        _act("act_prefill_t4096", 4096, 6912, 2560, 2, 4, "none", bias=False, residual=True),
        # backward of the epilogue: a small odd batch, and the 4096 tokens of a training step
        dict(name="act_grad_t509", op="act_grad", t=509, n_out=4864, experts=1, act="gelu"),
        dict(name="act_grad_t4096", op="act_grad", t=4096, n_out=6912, experts=16, act="relu2"),
        # one token routed to 8 of 64 experts
        _grouped("grouped_decode_r8", 8, 64, 56, 2048, 1408, 6, 8, "silu"),
        # a batch of 32 tokens, 8 experts each, over 64 experts
        _grouped("grouped_batch_r256", 256, 64, 3, 2048, 1408, 2, 4, "relu2", bias=True),
        # the rows of a training step, two experts idle
        _grouped("grouped_train_r16384", 16384, 32, 2, 2048, 2816, 6, 8, "relu2"),
        # dX and dW of a short, ragged step and of a training step
        _grouped("grouped_grad_r1000", 1000, 16, 1, 896, 1000, 8, 16, op="grouped_grad"),
        _grouped("grouped_grad_r8192", 8192, 16, 0, 2048, 1408, 6, 8, op="grouped_grad"),
        # the optimizer over a small adapter's tensors, and over twelve layers with 8-bit states
        dict(name="adamw_small_32", op="adamw", layers=4, d=200, f=520, bits=32, master=False),
        dict(name="adamw_layers_8", op="adamw", layers=12, d=896, f=4864, bits=8, master=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    n, m = rng.choice([(2, 4), (4, 8), (6, 8), (8, 16), (8, 8), (1, 4), (12, 16)])
    act = rng.choice(["none", "relu", "relu2", "silu", "gelu"])
    op = rng.choice(["act", "act", "act_grad", "grouped", "grouped", "grouped_grad", "adamw"])
    if op == "act":
        return dict(op=op, t=_log(rng, 1, 4096), k=128 * rng.randint(2, 54), n_out=_log(rng, 130, 2560), n=n, m=m,
                    act=act, bias=rng.random() < 0.6, residual=rng.random() < 0.5, save_z=rng.random() < 0.4)
    if op == "act_grad":
        return dict(op=op, t=_log(rng, 1, 4096), n_out=_log(rng, 130, 6912), experts=rng.choice([1, 1, 8, 33]),
                    act=act)
    if op == "adamw":
        return dict(op=op, layers=rng.randint(1, 12), d=_log(rng, 30, 896), f=_log(rng, 100, 4864),
                    bits=rng.choice([8, 32]), master=rng.random() < 0.5)
    experts = rng.choice([2, 5, 8, 16, 32])
    rows = _log(rng, 1, 8192)
    idle = max(experts - rows, rng.randint(0, experts // 2))
    c = dict(op=op, rows=rows, experts=experts, idle=idle, k=128 * rng.randint(2, 16), n_out=_log(rng, 130, 1408),
             n=n, m=m, act="none", bias=False)
    if op == "grouped":
        c.update(act=act, bias=rng.random() < 0.5)
    return c


def _adamw_sizes(c):
    one = [c["d"] * c["d"], c["d"] * c["f"], c["f"] * c["d"], c["f"], c["d"], 1]
    return one * c["layers"]


def work(c):
    op = c["op"]
    if op == "adamw":
        e = sum(_adamw_sizes(c))
        per = (10 if c["master"] else 4) + 2 + (4 if c["bits"] == 8 else 16)
        return {"bytes": per * e, "flops": 14 * e}
    if op == "act_grad":
        e = c["t"] * c["n_out"]
        return {"bytes": 6 * e + 4 * c["experts"] * c["n_out"], "flops": 8 * e}
    k, n_out, share = c["k"], c["n_out"], c["n"] / c["m"]
    weight = n_out * k * (2 * share + (0 if c["n"] == c["m"] else 1)) / 8
    if op == "act":
        rows, weights, biases = c["t"], weight, 1
    else:
        active = c["experts"] - c["idle"]
        rows, weights, biases = c["rows"], weight * active, active
    if op == "grouped_grad":
        moved = rows * (2 * n_out * 2 + k + 4 + 2 * k) + weights + 2 * c["experts"] * n_out * k
        return {"bytes": moved, "flops": 2 * rows * n_out * k * (1 + share)}
    outs = 1 + int(c.get("residual", False)) + int(c.get("save_z", False))
    moved = rows * (2 * k + 2 * n_out * outs) + weights + (4 * n_out * biases if c["bias"] else 0)
    return {"bytes": moved, "flops": 2 * rows * n_out * k * share}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _sizes(c, seed):
    """Rows of every expert: `idle` experts get none, the others at least one,
    the rest dealt out by uneven weights."""
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    order = torch.randperm(c["experts"], generator=g)
    active = order[: c["experts"] - c["idle"]]
    left = c["rows"] - active.numel()
    weight = torch.exp(0.5 * torch.randn(active.numel(), generator=g))
    take = torch.multinomial(weight, left, replacement=True, generator=g) if left else torch.zeros(0, dtype=torch.long)
    sizes = torch.zeros(c["experts"], dtype=torch.long)
    sizes[active] = 1 + torch.bincount(take, minlength=active.numel())
    return sizes


def _pack(w, n, m):
    """Latent weights [N, K] -> ternary int8 matrix, packed codes, keep bits
    and scale, in the packed layout of the library's header."""
    rows, k = w.shape
    mag = w.abs().float().view(rows, k // m, m)
    gamma = torch.clamp(w.abs().double().mean(), min=1e-5).float()
    rank = torch.zeros_like(mag, dtype=torch.int16)
    for j in range(m):
        other = mag[..., j : j + 1]
        earlier = torch.arange(m, device=w.device) > j
        rank += ((other > mag) | ((other == mag) & earlier)).to(torch.int16)
    keep = rank < n
    code = torch.clamp(torch.round(w.float().view(rows, k // m, m) / gamma), -1, 1).to(torch.int8) * keep
    ternary = code.view(rows, k).contiguous()
    place = torch.argsort((~keep).to(torch.int8), dim=-1, stable=True)[..., :n]
    kept = torch.gather(code, -1, place).view(rows, k // m * n).to(torch.int16) & 3
    row_bytes = (kept.shape[1] // 4 + 15) // 16 * 16
    quad = kept.view(rows, -1, 4)
    codes = torch.zeros(rows, row_bytes, dtype=torch.uint8, device=w.device)
    codes[:, : kept.shape[1] // 4] = (quad[..., 0] | quad[..., 1] << 2 | quad[..., 2] << 4 | quad[..., 3] << 6).to(
        torch.uint8)
    if n == m:
        return ternary, codes, None, gamma.view(1)
    bit = (2 ** torch.arange(8, device=w.device)).to(torch.int16)
    meta = torch.zeros(rows, (k // 8 + 15) // 16 * 16, dtype=torch.uint8, device=w.device)
    meta[:, : k // 8] = (keep.view(rows, k // 8, 8).to(torch.int16) * bit).sum(-1).to(torch.uint8)
    return ternary, codes, meta, gamma.view(1)


def _activations(rows, k, g):
    """Unit activations with a few channels ten times as large."""
    x = torch.randn(rows, k, device=DEV, generator=g)
    x[:, torch.randint(0, k, (max(1, k // 256),), device=DEV, generator=g)] *= 10.0
    return x.to(BF16)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(c)
    s.pop("name", None)
    op = c["op"]
    if op == "adamw":
        return _prepare_adamw(c, s, g)
    if op == "act_grad":
        s["z"] = torch.randn(c["t"], c["n_out"], device=DEV, generator=g).to(BF16)
        s["dy"] = (1e-3 * torch.randn(c["t"], c["n_out"], device=DEV, generator=g)).to(BF16)
        cuts = torch.randint(0, c["t"] + 1, (c["experts"] - 1,), device=DEV, generator=g).sort().values
        ends = torch.tensor([0, c["t"]], device=DEV)
        s["offsets"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
        s["expert"] = torch.bucketize(torch.arange(c["t"], device=DEV), s["offsets"][1:].long(), right=True)
        return s
    k, n_out = c["k"], c["n_out"]
    if op == "act":
        s["x"] = _activations(c["t"], k, g)
        s["ternary"], s["codes"], s["meta"], s["gamma"] = _pack(
            (0.02 * torch.randn(n_out, k, device=DEV, generator=g)).to(BF16), c["n"], c["m"])
        s["bias_v"] = 0.1 * torch.randn(n_out, device=DEV, generator=g) if c["bias"] else None
        s["residual_v"] = torch.randn(c["t"], n_out, device=DEV, generator=g).to(BF16) if c["residual"] else None
        s["y"] = torch.empty(c["t"], n_out, dtype=BF16, device=DEV)
        s["z"] = torch.empty(c["t"], n_out, dtype=BF16, device=DEV) if c["save_z"] else None
        return s
    e, rows = c["experts"], c["rows"]
    sizes = _sizes(c, seed)
    s["longest"] = int(sizes.max())
    s["sizes"] = sizes.to(DEV)
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long), sizes.cumsum(0)]).to(torch.int32).to(DEV)
    s["expert"] = torch.repeat_interleave(torch.arange(e, device=DEV), s["sizes"], output_size=rows)
    s["place"] = torch.arange(rows, device=DEV) - s["offsets"].long()[s["expert"]]
    packed = [_pack((0.02 * torch.randn(n_out, k, device=DEV, generator=g)).to(BF16), c["n"], c["m"])
              for _ in range(e)]
    s["ternary"] = torch.stack([p[0] for p in packed])
    s["codes"] = torch.stack([p[1] for p in packed])
    s["meta"] = None if c["n"] == c["m"] else torch.stack([p[2] for p in packed])
    s["gamma"] = torch.cat([p[3] for p in packed])
    x = _activations(rows, k, g)
    if op == "grouped_grad":
        s["dy"] = (1e-3 * torch.randn(rows, n_out, device=DEV, generator=g)).to(BF16)
        s["xq"], s["xs"] = _quantize(x)
        return s
    s["x"] = x
    s["bias_v"] = 0.1 * torch.randn(e, n_out, device=DEV, generator=g) if c["bias"] else None
    s["y"] = torch.empty(rows, n_out, dtype=BF16, device=DEV)
    return s


def _prepare_adamw(c, s, g):
    """Parameters, gradients and states as views of flat buffers, every tensor
    from a multiple of 256 elements on."""
    sizes = _adamw_sizes(c)
    starts, total = [], 0
    for e in sizes:
        starts.append(total)
        total += -(-e // BLOCK) * BLOCK
    used = torch.zeros(total, dtype=torch.bool, device=DEV)
    s["index"] = torch.arange(total, device=DEV, dtype=torch.int32)
    s["tensor"] = torch.zeros(total // BLOCK, dtype=torch.int64, device=DEV)
    for i, (e, at) in enumerate(zip(sizes, starts)):
        used[at : at + e] = True
        s["index"][at : at + -(-e // BLOCK) * BLOCK] -= at
        s["tensor"][at // BLOCK : (at + e + BLOCK - 1) // BLOCK] = i
    kind = F32 if c["master"] else BF16
    s["p"] = (0.02 * torch.randn(total, device=DEV, generator=g) * used).to(kind)
    s["copy"] = s["p"].to(BF16) if c["master"] else None
    s["g"] = (1e-3 * torch.randn(total, device=DEV, generator=g) * used).to(BF16)
    m = 3e-4 * torch.randn(total, device=DEV, generator=g) * used
    v = 1e-6 * torch.rand(total, device=DEV, generator=g) * used
    if c["bits"] == 8:
        s["m"], s["ms"] = _state8(m, torch.full((total,), 0.5, device=DEV))
        s["v"], s["vs"] = _state8(v.sqrt(), torch.full((total,), 0.5, device=DEV))
    else:
        s["m"], s["v"] = m, v
    s["step"] = torch.tensor([7, 0], dtype=torch.int32, device=DEV)

    def views(flat, per=1):
        return [flat[at // per : at // per + -(-e // per)] for e, at in zip(sizes, starts)]

    s["parts"] = {name: views(s[name], BLOCK if name in ("ms", "vs") else 1)
                  for name in ("p", "copy", "g", "m", "v", "ms", "vs") if s.get(name) is not None}
    return s


# --------------------------------------------------------------------------
# Plain form
# --------------------------------------------------------------------------
def _quantize(x):
    """Per-token absmax INT8: q = clamp(rint(x * (127 / s)), -127, 127)."""
    s = torch.clamp(x.float().abs().amax(dim=1), min=1e-5)
    q = torch.clamp(torch.round(x.float() * (127.0 / s)[:, None]), -127, 127)
    return q.to(torch.int8), s


def _f(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "relu2":
        return torch.clamp(z, min=0) * torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _df(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return 2 * torch.clamp(z, min=0)
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _padded(rows, s):
    """[R, C] rows sorted by expert -> [E, longest, C], zeros behind each expert's rows."""
    at = s["offsets"][:-1].long()[:, None] + torch.arange(s["longest"], device=DEV)
    valid = torch.arange(s["longest"], device=DEV) < s["sizes"][:, None]
    return rows[at.clamp(max=rows.shape[0] - 1)] * valid[..., None].to(rows.dtype)


def _plain_forward(s):
    q, xs = _quantize(s["x"])
    if s["op"] == "act":
        acc, gamma = q.float() @ s["ternary"].float().t(), s["gamma"]
    elif s["rows"] <= 16:
        acc = torch.bmm(s["ternary"][s["expert"]].float(), q.float()[:, :, None])[..., 0]
        gamma = s["gamma"][s["expert"]]
    else:
        acc = torch.bmm(_padded(q.float(), s), s["ternary"].float().transpose(1, 2))[s["expert"], s["place"]]
        gamma = s["gamma"][s["expert"]]
    z = acc * (gamma * xs / 127)[:, None]
    if s["bias_v"] is not None:
        z = z + (s["bias_v"] if s["op"] == "act" else s["bias_v"][s["expert"]])
    y = _f(z, s["act"])
    if s.get("residual_v") is not None:
        y = y + s["residual_v"].float()
    return [y.to(BF16)] + ([z.to(BF16)] if s.get("save_z") else [])


def _plain_act_grad(s):
    dz = s["dy"].float() * _df(s["z"].float(), s["act"])
    onehot = (s["expert"] == torch.arange(s["experts"], device=DEV)[:, None]).float()
    return [dz.to(BF16), onehot @ dz]


def _plain_grouped_grad(s):
    dy = _padded(s["dy"].float(), s)
    w = s["ternary"].float() * s["gamma"][:, None, None]
    xd = _padded(s["xq"].float() * (s["xs"] / 127)[:, None], s)
    dx = torch.bmm(dy, w)[s["expert"], s["place"]]
    dw = torch.bmm(dy.transpose(1, 2), xd)
    return [dx.to(BF16), dw.to(BF16)]


def _mix(x):
    """32-bit hash of whole numbers below 2^32, held in int64."""
    x = ((x ^ (x >> 16)) * HASH_A) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * HASH_B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _power(e):
    return ((e + 127) << 23).view(F32)


def _state8(x, u, root=False):
    """x -> e4m3 codes and one power of two per block of 256. Between two codes
    n and n + 1 (in steps of the grid at x) the upper one is taken with the
    probability that keeps x in expectation, or its square for a root, of which
    no positive value becomes zero; u is uniform in [0, 1)."""
    top = x.abs().view(-1, BLOCK).amax(dim=1)
    e = torch.clamp((top.view(torch.int32) >> 23) - 127, min=-100)
    y = (x.abs().view(-1, BLOCK) * _power(7 - e)[:, None]).view(-1)
    ey = torch.clamp((y.view(torch.int32) >> 23) - 127, min=-6)
    steps = y * _power(3 - ey)
    n = torch.floor(steps)
    up = u * (n + n + 1) < (steps - n) * (steps + n) if root else u < steps - n
    q = (n + up.float()) * _power(ey - 3)
    if root:
        q = torch.where(y > 0, torch.clamp(q, min=2.0**-9), q)
    return torch.copysign(q, x).to(torch.float8_e4m3fn), _power(e - 7)


def _plain_adamw(s):
    s["step"][0] += 1
    t = s["step"][0].double()
    a = (LR / (1 - BETA1**t)).float()
    c2 = (1 / torch.sqrt(1 - BETA2**t)).float()
    g = s["g"].float()
    if s["bits"] == 8:
        m0 = (s["m"].float().view(-1, BLOCK) * s["ms"][:, None]).view(-1)
        r0 = (s["v"].float().view(-1, BLOCK) * s["vs"][:, None]).view(-1)
        v0 = r0 * r0
    else:
        m0, v0 = s["m"], s["v"]
    m = BETA1 * m0 + (1 - BETA1) * g
    v = BETA2 * v0 + (1 - BETA2) * (g * g)
    r = torch.sqrt(v)
    p = s["p"].float() * (1 - LR * DECAY) - a * (m / (r * c2 + EPS))
    s["p"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    if s["bits"] == 8:
        key = _mix((SEED + s["step"][0].long() * HASH_A + s["tensor"] * HASH_B) & 0xFFFFFFFF)
        h = _mix((s["index"].long().view(-1, BLOCK) ^ key[:, None]).view(-1))
        m8, ms = _state8(m, (h & 0xFFFF).float() * 2.0**-16)
        v8, vs = _state8(r, (h >> 16).float() * 2.0**-16, root=True)
        s["m"].copy_(m8)
        s["ms"].copy_(ms)
        s["v"].copy_(v8)
        s["vs"].copy_(vs)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_out(s)


def _adamw_out(s):
    return {name: s[name] for name in ("p", "copy", "m", "ms", "v", "vs") if s.get(name) is not None}


# --------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------
def _weights(s, sbn):
    """The packed weights as the library's handle, built on first use."""
    if "handle" not in s:
        args = (s["codes"], s["meta"], s["gamma"], s["n_out"], s["k"], s["n"], s["m"])
        s["handle"] = sbn.PackedWeights(*args) if s["op"] == "act" else sbn.PackedExperts(*args, s["experts"])
    return s["handle"]


def _own(s):
    from sparse_linear_layers_fwd_b200 import sbn

    op = s["op"]
    if op == "act":
        sbn.bitlinear_x_act(s["x"], _weights(s, sbn), bias=s["bias_v"], act=s["act"], residual=s["residual_v"],
                            out=s["y"], out_z=s["z"])
        return [s["y"]] + ([s["z"]] if s["save_z"] else [])
    if op == "act_grad":
        return list(sbn.act_grad(s["dy"], s["z"], s["act"], offsets=s["offsets"]))
    if op == "grouped":
        return [sbn.bitlinear_grouped_x(s["x"], s["offsets"], _weights(s, sbn), bias=s["bias_v"], act=s["act"],
                                        out=s["y"])]
    if op == "grouped_grad":
        return [sbn.bitlinear_grouped_grad_x(s["dy"], s["offsets"], _weights(s, sbn)),
                sbn.bitlinear_grouped_grad_w(s["dy"], s["xq"], s["xs"], s["offsets"])]
    if "handle" not in s:
        q = s["parts"]
        s["handle"] = opt = sbn.AdamW(q["p"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
                                      state_bits=s["bits"], copies=q.get("copy"), seed=SEED)
        opt.m, opt.v, opt.m_scales, opt.v_scales = q["m"], q["v"], q.get("ms"), q.get("vs")
        opt.step_state = s["step"]
    s["handle"].step(s["parts"]["g"])
    return _adamw_out(s)


def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op in ("act", "grouped"):
        return _plain_forward(s)
    return {"act_grad": _plain_act_grad, "grouped_grad": _plain_grouped_grad, "adamw": _plain_adamw}[op](s)


# --------------------------------------------------------------------------
# The definitions in 64 bits, row by row and expert by expert
# --------------------------------------------------------------------------
def _exact_f(z, act):
    if act == "none":
        return z
    if act in ("relu", "relu2"):
        return torch.where(z > 0, z if act == "relu" else z * z, torch.zeros_like(z))
    if act == "silu":
        return z * torch.special.expit(z)
    return z * torch.special.ndtr(z)


def _exact_df(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act in ("relu", "relu2"):
        return torch.where(z > 0, torch.ones_like(z) if act == "relu" else 2 * z, torch.zeros_like(z))
    if act == "silu":
        sig = torch.special.expit(z)
        return sig + z * sig * torch.special.expit(-z)
    return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "adamw":
        t = int(s["step"][0]) + 1
        g = s["g"].double()
        if c["bits"] == 8:
            m0 = s["m"].double() * s["ms"].double().repeat_interleave(BLOCK)
            v0 = (s["v"].double() * s["vs"].double().repeat_interleave(BLOCK)) ** 2
        else:
            m0, v0 = s["m"].double(), s["v"].double()
        m, v = m0 + (1 - BETA1) * (g - m0), v0 + (1 - BETA2) * (g**2 - v0)
        step = (m / (1 - BETA1**t)) / ((v / (1 - BETA2**t)).sqrt() + EPS)
        p = s["p"].double() - LR * DECAY * s["p"].double() - LR * step
        out = {"p": p, "copy": p if c["master"] else None}
        # codes of 8 bits hang on the remainder at their border: no value in 64 bits
        eight = c["bits"] == 8
        out.update({"m": None if eight else m, "v": None if eight else v})
        if eight:
            out.update({"ms": None, "vs": None})
        return {k: v for k, v in out.items() if s.get(k) is not None}
    if op == "act_grad":
        dz = s["dy"].double() * _exact_df(s["z"].double(), c["act"])
        ends = s["offsets"].tolist()
        return [dz, torch.stack([dz[a:b].sum(0) for a, b in zip(ends[:-1], ends[1:])])]
    spans = [(0, c["t"])] if op == "act" else list(zip(s["offsets"].tolist()[:-1], s["offsets"].tolist()[1:]))
    weight = s["ternary"].view(len(spans), c["n_out"], c["k"])
    if op == "grouped_grad":
        xd = s["xq"].double() * s["xs"].double()[:, None] / 127
        dx, dw = torch.zeros_like(xd), torch.zeros(weight.shape, dtype=F64, device=DEV)
        for i, (a, b) in enumerate(spans):
            dx[a:b] = s["dy"][a:b].double() @ weight[i].double() * s["gamma"][i].double()
            dw[i] = s["dy"][a:b].double().t() @ xd[a:b]
        return [dx, dw]
    # the quantizer's two roundings in 32 bits are its definition
    scale = s["x"].abs().amax(dim=1).float().clamp(min=1e-5)
    mult = torch.full_like(scale, 127.0) / scale
    q = (s["x"].float() * mult[:, None]).round().clamp(-127, 127).double()
    z = torch.zeros(q.shape[0], c["n_out"], dtype=F64, device=DEV)
    for i, (a, b) in enumerate(spans):
        z[a:b] = q[a:b] @ weight[i].double().t() * s["gamma"][i].double() * scale[a:b].double()[:, None] / 127
        if s["bias_v"] is not None:
            z[a:b] += s["bias_v"].view(len(spans), -1)[i].double()
    y = _exact_f(z, c["act"])
    if s.get("residual_v") is not None:
        y = y + s["residual_v"].double()
    return [y] + ([z] if c.get("save_z") else [])
