"""The layer's epilogue and the grouped layer against 64-bit references.

Reference: oracle codes, scales and INT8 activations (checked bit for bit by
the parity tests), everything after the integer accumulators in float64.

Tolerances, u = 2^-24 (half a step of fp32), h = 2^-8 (of bf16):
  z   acc (exact below 2^24, else 1 u) times a factor of three roundings, one
      product, one sum: within 6 u of Z = |acc gamma s / 127| + |bias|;
  f   relu2 doubles a relative error (its slope is 2 |z|); the slopes of the
      others are below 1.13. Their own evaluation: relu2 one product; silu an
      exponential whose argument -z log2 e carries two roundings (2 |z| u of the
      result, by d 2^x = 2^x ln 2 dx) and 4 u of its own, a sum, a reciprocal of
      4 u, a product: (2 |z| + 12) u |f|; gelu the rational approximation of
      Abramowitz and Stegun 7.1.26, 1.5e-7 of erfc and so 0.75e-7 of Phi, with
      at most 2^-23 more of the fp32 evaluation (Phi <= 1, five products and
      sums of terms below 2, two special functions; the exponential's argument
      error z^2 u of a result below exp(-z^2 / 2) stays below u): 2e-7 |z|;
  y   one sum and one rounding to bf16:
      h |y| + (1 + h) (6 u slope Z + error of f + u |y|).
  dX, dW  sums of n products exact in fp32, accumulated in fp32 in any order:
      n u times the sum of |products|, doubled for the tensor core's alignment
      of addends, plus h of the result. dW's factor a = dY s / 127 is rounded to
      fp16 after a power of two per feature brought the largest |a| of its column
      to [2^14, 2^15): half a step of fp16 is 2^-11 of a, or 2^-25 absolute
      below 2^-14, that is at most 2^-39 of the column's largest; with the two
      roundings of a itself 2^-11 + 4 u, plus 2^-39 max |a| sum |x|.
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from sparse_linear_layers_fwd_b200 import synth

U, H = 2.0 ** -24, 2.0 ** -8
ACT_NAMES = ["none", "relu", "relu2", "silu", "gelu"]
PATTERNS = [(1, 4), (2, 4), (3, 4), (4, 4), (2, 8), (4, 8), (6, 8), (8, 8), (4, 16), (8, 16), (12, 16), (16, 16)]
A, MIS = 0x10000, 0x10008


def _sbn():
    from sparse_linear_layers_fwd_b200 import sbn
    return sbn


def f64(act, z):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "relu2":
        return torch.clamp(z, min=0) ** 2
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z


def df64(act, z):
    if act == "relu":
        return (z > 0).double()
    if act == "relu2":
        return 2 * torch.clamp(z, min=0)
    if act == "silu":
        s = torch.special.expit(z)
        return s * (1 + z * torch.special.expit(-z))
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    return torch.ones_like(z)


@pytest.mark.parametrize("act", ACT_NAMES)
def test_reference_derivative_against_differences(act):
    z = torch.linspace(-6, 6, 97, dtype=torch.float64) + 0.013
    e = 1e-6
    d = (f64(act, z + e) - f64(act, z - e)) / (2 * e)
    assert torch.allclose(d, df64(act, z), atol=1e-8)


# --------------------------------------------------------------------------
# CPU: argument checks of the C entries
# --------------------------------------------------------------------------
def act_call(lib, xq=A, xs=A, t=64, k=256, n_out=64, n=2, m=4, codes=A, meta=A, gamma=A, bias=A, act=0, res=A, z=A, y=A,
             ws=A, wsb=1 << 30):
    return lib.sbn_bitlinear_act(xq, xs, t, k, n_out, n, m, codes, meta, gamma, bias, act, res, z, y, ws, wsb, None)


def x_act_call(lib, x=A, t=64, k=256, n_out=64, n=2, m=4, codes=A, meta=A, gamma=A, bias=None, act=0, res=None, z=None,
               y=A, xq=None, xs=None, ws=A, wsb=1 << 30):
    return lib.sbn_bitlinear_x_act(x, t, k, n_out, n, m, codes, meta, gamma, bias, act, res, z, y, xq, xs, ws, wsb, None)


def grp_call(lib, xq=A, xs=A, rows=64, off=A, experts=4, k=256, n_out=64, n=2, m=4, codes=A, meta=A, gamma=A, bias=None,
             act=0, res=None, z=None, y=A):
    return lib.sbn_bitlinear_grouped(xq, xs, rows, off, experts, k, n_out, n, m, codes, meta, gamma, bias, act, res, z,
                                     y, None)


def grp_x_call(lib, x=A, rows=64, off=A, experts=4, k=256, n_out=64, n=2, m=4, codes=A, meta=A, gamma=A, y=A, xq=None,
               xs=None, ws=A, wsb=1 << 30):
    return lib.sbn_bitlinear_grouped_x(x, rows, off, experts, k, n_out, n, m, codes, meta, gamma, None, 0, None, None,
                                       y, xq, xs, ws, wsb, None)


def test_forward_validation(sbn_lib):
    lib = sbn_lib
    for call in (act_call, grp_call):
        for name in ("xq", "xs", "codes", "meta", "gamma", "y"):
            assert call(lib, **{name: None}) == 1, (call, name)
        assert call(lib, n=3, m=8) == 3
        assert call(lib, k=200) == 2
        assert call(lib, n_out=0) == 2
        assert call(lib, act=5) == 2
        assert call(lib, act=-1) == 2
        for name in ("xq", "codes", "meta", "y", "z", "res"):
            assert call(lib, **{name: MIS}) == 4, (call, name)
        for name in ("xs", "gamma", "bias"):
            assert call(lib, **{name: A + 2}) == 4, (call, name)
        assert call(lib, n_out=1 << 20, k=1 << 12) == 2
    assert act_call(lib, t=0) == 2
    assert act_call(lib, wsb=100) == 5
    assert act_call(lib, ws=MIS) == 4
    assert x_act_call(lib, x=None) == 1
    assert x_act_call(lib, x=MIS) == 4
    assert x_act_call(lib, xq=MIS) == 4
    assert x_act_call(lib, t=1 << 20, k=1 << 12) == 2
    assert grp_call(lib, off=None) == 1
    assert grp_call(lib, off=A + 2) == 4
    assert grp_call(lib, rows=0) == 2
    assert grp_call(lib, experts=0) == 2
    assert grp_call(lib, experts=1025) == 2
    assert grp_x_call(lib, x=None) == 1
    assert grp_x_call(lib, off=None) == 1
    assert grp_x_call(lib, x=MIS) == 4
    assert lib.sbn_bitlinear_grouped_x_workspace_bytes(64, 256) == 64 * 256 + 64 * 4
    assert lib.sbn_bitlinear_grouped_x_workspace_bytes(0, 256) == 0


def test_backward_validation(sbn_lib):
    lib = sbn_lib

    def ag(dy=A, z=A, rows=64, off=A, e=4, n_out=64, act=1, dz=A, db=A):
        return lib.sbn_act_grad(dy, z, rows, off, e, n_out, act, dz, db, None)

    def gx(dy=A, rows=64, off=A, e=4, k=256, n_out=64, n=2, m=4, codes=A, meta=A, gamma=A, dx=A, ws=None,
           wsb=0):
        return lib.sbn_bitlinear_grouped_grad_x(dy, rows, off, e, k, n_out, n, m, codes, meta, gamma, dx, ws, wsb, None)

    def gw(dy=A, xq=A, xs=A, rows=64, off=A, e=4, k=256, n_out=64, dw=A, ws=A, wsb=1 << 30):
        return lib.sbn_bitlinear_grouped_grad_w(dy, xq, xs, rows, off, e, k, n_out, dw, ws, wsb, None)
    for name in ("dy", "z", "dz"):
        assert ag(**{name: None}) == 1
        assert ag(**{name: MIS}) == 4
    assert ag(off=None) == 2              # several groups need offsets
    assert ag(act=9) == 2 and ag(rows=0) == 2 and ag(e=0) == 2 and ag(e=2000) == 2 and ag(n_out=0) == 2
    assert ag(db=A + 2) == 4 and ag(off=A + 2) == 4
    for name in ("dy", "off", "codes", "meta", "gamma", "dx"):
        assert gx(**{name: None}) == 1
    assert gx(n=5, m=8) == 3 and gx(k=100) == 2 and gx(rows=0) == 2 and gx(e=1025) == 2
    assert gx(dy=MIS) == 4 and gx(dx=MIS) == 4
    assert lib.sbn_bitlinear_grouped_grad_x_workspace_bytes(64, 64) == 0
    assert lib.sbn_bitlinear_grouped_grad_x_workspace_bytes(64, 65) == 64 * 72 * 2
    assert lib.sbn_bitlinear_grouped_grad_x_workspace_bytes(0, 65) == 0
    assert gx(n_out=65) == 5 and gx(n_out=65, ws=A, wsb=64 * 72 * 2 - 1) == 5 and gx(n_out=65, ws=MIS, wsb=1 << 30) == 4
    for name in ("dy", "xq", "xs", "off", "dw"):
        assert gw(**{name: None}) == 1
    assert gw(k=100) == 2 and gw(n_out=0) == 2 and gw(e=0) == 2
    assert gw(xq=MIS) == 4 and gw(dw=MIS) == 4 and gw(ws=MIS) == 4
    need = lib.sbn_bitlinear_grouped_grad_w_workspace_bytes(64, 4, 256, 64)
    rows = (64 + 4 * 63) // 64 * 64       # every expert's rows end a block of 64
    assert need == rows * 64 * 2 + rows * 256 * 2 + 4 * 64 * 4
    assert gw(wsb=need - 1) == 5 and gw(ws=None) == 5
    # features at a pitch of eight, the last array rounded up to 16 bytes
    assert lib.sbn_bitlinear_grouped_grad_w_workspace_bytes(64, 4, 256, 65) == rows * 72 * 2 + rows * 256 * 2 + 4 * 65 * 4
    assert lib.sbn_bitlinear_grouped_grad_w_workspace_bytes(64, 4, 100, 64) == 0


def test_acts_of_binding_and_header_agree():
    import re
    from pathlib import Path
    text = (Path(__file__).resolve().parents[1] / "include" / "sbn.h").read_text()
    got = {k.lower(): int(v) for k, v in re.findall(r"#define SBN_ACT_([A-Z0-9]+) (\d)", text)}
    assert got == _sbn().ACTS
    with pytest.raises(ValueError):
        _sbn()._act("tanh")


# --------------------------------------------------------------------------
# GPU
# --------------------------------------------------------------------------
gpu = pytest.mark.gpu


def bits_to_dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


class Layer:
    """E experts of one shape: latent weights, packed weights, dense codes."""

    def __init__(self, experts, n_out, k, n, m, tag):
        sbn = _sbn()
        ws = [synth.latent_weights(n_out, k, seed=41 + e, tag=f"{tag}{n}{m}") for e in range(experts)]
        self.latent = torch.stack([bits_to_dev(w) for w in ws])
        self.packed = sbn.quantize_experts(self.latent, n, m)
        ref = [oracle.quantize_weights(w, n, m) for w in ws]
        for e, r in enumerate(ref):
            assert np.array_equal(self.packed.codes[e].cpu().numpy(), r[0])
            if n != m:
                assert np.array_equal(self.packed.meta[e].cpu().numpy(), r[1])
        self.gamma = torch.tensor([float(r[2]) for r in ref], dtype=torch.float64, device="cuda")
        assert torch.equal(self.packed.gamma.double(), self.gamma)
        self.dense = torch.stack([torch.from_numpy(np.asarray(r[4], dtype=np.float64)).cuda() for r in ref])


def acts_of(rows, k, tag):
    bits = synth.activations(rows, k, seed=43, tag=f"ff{tag}", outlier_channels=1)
    q, s = oracle.quantize_acts(bits)
    return bits_to_dev(bits), torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()


def reference(layer, q, s, spans, bias, act, residual):
    """(y, tolerance of y, z, tolerance of z) in float64; zero outside the spans."""
    rows, n_out = q.shape[0], layer.dense.shape[1]
    zero = lambda: torch.zeros(rows, n_out, dtype=torch.float64, device="cuda")  # noqa: E731
    z, mag = zero(), zero()
    for e, (a, b) in enumerate(spans):
        p = (q[a:b].double() @ layer.dense[e].T) * (layer.gamma[e] * s[a:b].double() / 127)[:, None]
        z[a:b], mag[a:b] = p, p.abs()
        if bias is not None:
            z[a:b] += bias.view(len(spans), n_out)[e].double()
            mag[a:b] += bias.view(len(spans), n_out)[e].double().abs()
    f = f64(act, z)
    slope = 2 * z.abs() + 1 if act == "relu2" else 1.13
    y = f if residual is None else f + residual.double()
    own = {"silu": (2 * z.abs() + 12) * U * f.abs(), "gelu": 2e-7 * z.abs()}.get(act, 2 * U * f.abs())
    err = 6 * U * slope * mag + own + U * y.abs()
    return y, H * y.abs() + (1 + H) * err, z, H * z.abs() + (1 + H) * 6 * U * mag


def close(got, ref, tol, what):
    bad = (got.double() - ref).abs() > tol + 1e-38
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def epilogue_inputs(rows, n_out, experts, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bias = 0.3 * torch.randn((experts, n_out) if experts else (n_out,), device="cuda", generator=g)
    res = torch.randn(rows, n_out, device="cuda", generator=g).to(torch.bfloat16)
    return bias, res


def clean(sbn):
    torch.cuda.synchronize()
    assert sbn.get_device_error() == 0


# rows, K, N_out, pattern: the decode kernel (1 to 16 rows, K below one item,
# one tile, rows whose activations or weights do not fit it), the pair kernel's
# three tiles, ragged everything, N_out that is no multiple of 8
ACT_CASES = [
    (1, 128, 16, 6, 8), (1, 2560, 6912, 6, 8), (5, 384, 257, 2, 4), (8, 11008, 100, 6, 8), (9, 512, 33, 8, 16),
    (16, 1024, 130, 4, 8), (16, 11008, 72, 2, 4), (17, 384, 264, 6, 8), (100, 512, 257, 6, 8), (225, 384, 136, 2, 4),
    (300, 640, 520, 8, 8), (1000, 384, 4000, 6, 8), (33, 256, 64, 12, 16),
]


@gpu
@pytest.mark.parametrize("case", ACT_CASES, ids=["t%d_k%d_n%d_%dof%d" % c for c in ACT_CASES])
def test_act_routes(sbn_lib, cuda_ok, case):
    sbn = _sbn()
    t, k, n_out, n, m = case
    layer = Layer(1, n_out, k, n, m, f"act{case}")
    w = layer.packed.expert(0)
    x, q, s = acts_of(t, k, str(case))
    bias, res = epilogue_inputs(t, n_out, 0)
    plans = [("gelu", bias, res, True), ("relu2", bias, None, False), ("none", None, res, False),
             ("silu", None, None, True), ("relu", bias, res, True)]
    for act, b, r, want_z in plans:
        y, ytol, z, ztol = reference(layer, q, s, [(0, t)], b, act, r)
        outs = []
        for route in ("x", "ws", "no_ws"):
            oz = torch.empty(t, n_out, dtype=torch.bfloat16, device="cuda") if want_z else None
            if route == "x":
                oq, os_ = torch.empty_like(q), torch.empty_like(s)
                got = sbn.bitlinear_x_act(x, w, bias=b, act=act, residual=r, out_z=oz, out_q=oq, out_s=os_)
                assert torch.equal(oq, q) and torch.equal(os_, s)
            else:
                got = sbn.bitlinear_act(q, s, w, bias=b, act=act, residual=r, out_z=oz,
                                        workspace=None if route == "ws" else False)
            clean(sbn)
            close(got, y, ytol, f"{act} {route}")
            if want_z:
                close(oz, z, ztol, f"z {act} {route}")
            outs.append((got, oz))
        # integer accumulators and one fp32 epilogue: every route gives the same bits
        for got, oz in outs[1:]:
            assert torch.equal(got, outs[0][0])
            assert oz is None or torch.equal(oz, outs[0][1])
    # without an epilogue it is bitlinear, bit for bit; and the residual in place
    assert torch.equal(sbn.bitlinear_act(q, s, w), sbn.bitlinear(q, s, w))
    inplace = res.clone()
    sbn.bitlinear_act(q, s, w, bias=bias, act="silu", residual=inplace, out=inplace)
    assert torch.equal(inplace, sbn.bitlinear_act(q, s, w, bias=bias, act="silu", residual=res))
    clean(sbn)


@gpu
@pytest.mark.parametrize("nm", PATTERNS, ids=["%dof%d" % p for p in PATTERNS])
def test_every_pattern(sbn_lib, cuda_ok, nm):
    """Forward (decode and tensor-core), dX and dW of every pattern."""
    sbn = _sbn()
    n, m = nm
    k, n_out = 640, 200
    layer = Layer(3, n_out, k, n, m, "pat")
    for sizes in ((3, 0, 5), (150, 1, 70)):
        off = np.concatenate([[0], np.cumsum(sizes)])
        spans = list(zip(off[:-1], off[1:]))
        rows = int(off[-1])
        x, q, s = acts_of(rows, k, f"pat{nm}{rows}")
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        y, ytol, _, _ = reference(layer, q, s, spans, None, "gelu", None)
        close(sbn.bitlinear_grouped(q, s, o, layer.packed, act="gelu"), y, ytol, f"{sizes}")
        dy = (1e-2 * torch.randn(rows, n_out, device="cuda")).to(torch.bfloat16)
        check_grads(layer, dy, q, s, spans, o)
    clean(sbn)


def dw_reference(d, xd):
    """dW of one expert and its tolerance, from its float64 rows of dY and Xd."""
    ref, mag = d.T @ xd, d.abs().T @ xd.abs()
    n = d.shape[0]
    tol = (2 * n + 8) * U * mag + 2.0 ** -11 * mag   # fp32 sums of products of a factor rounded to fp16
    if n:   # and of factors too small for fp16's normal range
        tol = tol + 2.0 ** -39 * d.abs().amax(dim=0)[:, None] * xd.abs().amax() * n
    return ref, H * ref.abs() + (1 + H) * tol


def check_grads(layer, dy, q, s, spans, o):
    sbn = _sbn()
    dx = sbn.bitlinear_grouped_grad_x(dy, o, layer.packed)
    dw = sbn.bitlinear_grouped_grad_w(dy, q, s, o)
    clean(sbn)
    xd = q.double() * s.double()[:, None] / 127
    n_out = dy.shape[1]
    for e, (a, b) in enumerate(spans):
        wd = layer.dense[e] * layer.gamma[e]
        d = dy[a:b].double()
        ref, mag = d @ wd, d.abs() @ wd.abs()
        close(dx[a:b], ref, H * ref.abs() + (1 + H) * (2 * n_out + 4) * U * mag, f"dx {e}")
        close(dw[e], *dw_reference(d, xd[a:b]), f"dw {e}")
    return dx, dw


# sizes per expert, K, N_out, pattern
GRP_CASES = [
    ((1,), 128, 16, 6, 8),
    ((0, 0, 1), 256, 40, 2, 4),
    ((2, 0, 6, 0, 0, 8), 384, 257, 6, 8),
    ((16,), 1024, 130, 8, 8),
    ((4, 4, 4, 4), 2048, 1408, 6, 8),
    ((0, 17, 0), 256, 100, 6, 8),
    ((1, 31, 32, 33, 0, 96, 97), 384, 264, 2, 4),
    ((255, 256, 257), 256, 129, 4, 8),
    ((600, 0, 3, 1), 512, 384, 6, 8),
    ((7,) * 40, 256, 72, 8, 16),
    ((0,) * 900 + (1, 1, 40) + (0,) * 121, 128, 24, 1, 4),
    ((0,) * 1000 + (2, 1) + (0,) * 22, 128, 24, 3, 4),
    # several tiles for each CTA: of one, three and five blocks of positions
    ((33,) * 40, 128, 2000, 6, 8),
    ((40,) * 30, 384, 1500, 2, 4),
    ((700, 0, 450, 900), 640, 2100, 8, 8),
]


@gpu
@pytest.mark.parametrize("case", GRP_CASES, ids=[f"e{len(c[0])}_r{sum(c[0])}_k{c[1]}_n{c[2]}_{c[3]}of{c[4]}" for c in GRP_CASES])
@pytest.mark.parametrize("head,tail", [(0, 0), (3, 5)])
def test_grouped(sbn_lib, cuda_ok, case, head, tail):
    """Ragged sizes, experts without rows, rows before the first and behind
    the last expert (left as they were)."""
    sbn = _sbn()
    sizes, k, n_out, n, m = case
    if head and len(sizes) > 500 and sum(sizes) < 16:
        head, tail = 1, 1   # stays in the decode kernel
    off = head + np.concatenate([[0], np.cumsum(sizes)])
    spans = list(zip(off[:-1].tolist(), off[1:].tolist()))
    rows = int(off[-1]) + tail
    few = Layer(min(len(sizes), 8), n_out, k, n, m, "grp")   # expert e uses layer e % 8
    pick = torch.arange(len(sizes), device="cuda") % few.packed.experts
    layer = Layer.__new__(Layer)
    layer.packed = sbn.PackedExperts(few.packed.codes[pick].contiguous(),
                                     None if n == m else few.packed.meta[pick].contiguous(),
                                     few.packed.gamma[pick].contiguous(), n_out, k, n, m, len(sizes))
    layer.dense, layer.gamma = [few.dense[i] for i in pick.tolist()], few.gamma[pick]

    class Dense(list):
        shape = (len(sizes), n_out, k)
    layer.dense = Dense(layer.dense)
    x, q, s = acts_of(rows, k, str(case)[:40])
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    bias, res = epilogue_inputs(rows, n_out, len(sizes))
    inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
    inside[int(off[0]):int(off[-1])] = True
    for act, b, r in (("silu", bias, res), ("relu2", None, None)):
        y, ytol, z, ztol = reference(layer, q, s, spans, b, act, r)
        for fused in (False, True):
            out = torch.full((rows, n_out), 77.0, dtype=torch.bfloat16, device="cuda")
            oz = torch.full((rows, n_out), 78.0, dtype=torch.bfloat16, device="cuda")
            if fused:
                sbn.bitlinear_grouped_x(x, o, layer.packed, bias=b, act=act, residual=r, out=out, out_z=oz)
            else:
                sbn.bitlinear_grouped(q, s, o, layer.packed, bias=b, act=act, residual=r, out=out, out_z=oz)
            clean(sbn)
            assert (out[~inside] == 77.0).all() and (oz[~inside] == 78.0).all()
            close(out[inside], y[inside], ytol[inside], f"{act} {fused}")
            close(oz[inside], z[inside], ztol[inside], f"z {act} {fused}")
    # backward, rows outside untouched
    dy = (1e-2 * torch.randn(rows, n_out, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))).to(
        torch.bfloat16)
    dx = torch.full((rows, k), 79.0, dtype=torch.bfloat16, device="cuda")
    sbn.bitlinear_grouped_grad_x(dy, o, layer.packed, out=dx)
    clean(sbn)
    assert (dx[~inside] == 79.0).all()
    dx2, dw = check_grads(layer, dy, q, s, spans, o)
    assert torch.equal(dx[inside], dx2[inside])
    for e, n_e in enumerate(sizes):
        if n_e == 0:
            assert (dw[e] == 0).all()


@gpu
@pytest.mark.parametrize("rows,experts", [(10, 5), (200, 5)])
def test_offsets_out_of_order_stay_in_bounds(sbn_lib, cuda_ok, rows, experts):
    """Offsets that decrease, start below zero or end behind the rows are
    clamped on the device: nothing outside the outputs changes, and a call with
    the clamped offsets gives the same."""
    from test_canaries import Guarded
    sbn = _sbn()
    k, n_out = 256, 136
    layer = Layer(experts, n_out, k, 6, 8, "bad")
    x, q, s = acts_of(rows, k, f"bad{rows}")
    dy = (1e-2 * torch.randn(rows, n_out, device="cuda")).to(torch.bfloat16)
    for bad in ([-5, 3, 1, 2 ** 31 - 1, 7, 2], [rows + 9] * (experts + 1), [0, 4, 2, 6, 5, rows + 100],
                [-(2 ** 31)] * experts + [rows]):
        good = np.maximum.accumulate(np.clip(np.array(bad, dtype=np.int64), 0, rows))
        res = []
        for off in (bad, good):
            g = Guarded()
            o = torch.tensor(np.array(off, dtype=np.int64), device="cuda").to(torch.int32)
            y, dx = g.tensor((rows, n_out), torch.bfloat16), g.tensor((rows, k), torch.bfloat16)
            dw = g.tensor((experts, n_out, k), torch.bfloat16)
            y.fill_(1.0), dx.fill_(1.0)
            sbn.bitlinear_grouped(q, s, o, layer.packed, act="relu", out=y)
            sbn.bitlinear_grouped_grad_x(dy, o, layer.packed, out=dx)
            sbn.bitlinear_grouped_grad_w(dy, q, s, o, out=dw)
            g.check()
            res.append((y, dx, dw))
        assert all(torch.equal(a, b) for a, b in zip(*res)), bad


@gpu
@pytest.mark.parametrize("act", ACT_NAMES)
@pytest.mark.parametrize("rows,n_out,sizes", [(1, 1, None), (37, 264, None), (300, 129, (0, 250, 0, 50)),
                                              (1500, 200, (1000, 1, 499)), (70, 4864, (64, 0, 3))])
def test_act_grad(sbn_lib, cuda_ok, act, rows, n_out, sizes):
    """dz within one bf16 rounding and the derivative's evaluation: silu's
    s (1 + z (1 - s)) has s within (2 |z| + 9) u of itself, so the bracket is
    within (|z| + 1) (2 |z| + 12) u; gelu's Phi is within 2e-7 and z phi within
    (z^2 + 8) u |z phi| < 8 u; times |dy|. dbias within the fp32 sum's n u of the
    sum of |dz| plus the terms' own errors; the same bits on every run."""
    from test_canaries import Guarded
    sbn = _sbn()
    g = torch.Generator(device="cuda").manual_seed(rows)
    dy = torch.randn(rows, n_out, device="cuda", generator=g).to(torch.bfloat16)
    z = (3 * torch.randn(rows, n_out, device="cuda", generator=g)).to(torch.bfloat16)
    z[0, 0] = 0.0
    o, spans = None, [(0, rows)]
    if sizes is not None:
        off = np.concatenate([[0], np.cumsum(sizes)])
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        spans = list(zip(off[:-1].tolist(), off[1:].tolist()))
    inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
    inside[spans[0][0]:spans[-1][1]] = True
    gd = Guarded()
    dz = gd.tensor((rows, n_out), torch.bfloat16)
    dz.fill_(5.0)
    db = gd.tensor((n_out,) if o is None else (len(sizes), n_out), torch.float32)
    sbn.act_grad(dy, z, act, offsets=o, out=dz, out_bias=db)
    gd.check()
    ref = dy.double() * df64(act, z.double())
    az = z.double().abs()
    own = {"silu": (az + 2) * (2 * az + 12) * U, "gelu": 2e-7 + 8 * U + 0 * az}.get(act, 2 * U * (2 * az + 1))
    e = dy.double().abs() * own
    close(dz[inside], ref[inside], (H * ref.abs() + (1 + H) * e)[inside], "dz")
    assert (dz[~inside] == 5.0).all()
    for i, (a, b) in enumerate(spans):
        want = ref[a:b].sum(0)
        tol = (b - a) * U * ref[a:b].abs().sum(0) + 2 * e[a:b].sum(0)
        close(db.view(len(spans), n_out)[i], want, tol, f"dbias {i}")
    again, db2 = sbn.act_grad(dy.clone(), z, act, offsets=o)
    assert torch.equal(db2, db) and torch.equal(again[inside], dz[inside])
    inplace = dy.clone()
    _, none = sbn.act_grad(inplace, z, act, offsets=o, out=inplace, out_bias=False)
    assert none is None and torch.equal(inplace[inside], dz[inside])
    clean(sbn)


@gpu
def test_canaries_of_the_new_calls(sbn_lib, cuda_ok):
    from test_canaries import Guarded
    sbn = _sbn()
    for t, k, n_out, n, m in [(5, 384, 257, 6, 8), (16, 640, 136, 2, 4), (100, 512, 257, 6, 8), (225, 384, 136, 2, 4),
                              (300, 640, 520, 4, 8)]:
        layer = Layer(2, n_out, k, n, m, "can")
        x, q, s = acts_of(t, k, f"can{t}")
        bias, res = epilogue_inputs(t, n_out, 0)
        g = Guarded()
        new = lambda *shape: g.tensor(shape, torch.bfloat16)  # noqa: E731
        sbn.bitlinear_x_act(x, layer.packed.expert(0), bias=bias, act="gelu", residual=res, out=new(t, n_out),
                            out_z=new(t, n_out), out_q=g.tensor((t, k), torch.int8), out_s=g.tensor((t,), torch.float32),
                            workspace=g.tensor((sbn.bitlinear_x_workspace_bytes(t, k, n_out),), torch.uint8))
        sbn.bitlinear_act(q, s, layer.packed.expert(1), act="relu2", out=new(t, n_out), workspace=False)
        o = torch.tensor([0, t // 3, t], dtype=torch.int32, device="cuda")
        nb = int(sbn.lib().sbn_bitlinear_grouped_x_workspace_bytes(t, k))
        sbn.bitlinear_grouped_x(x, o, layer.packed, act="silu", out=new(t, n_out), out_z=new(t, n_out),
                                workspace=g.tensor((nb,), torch.uint8))
        sbn.bitlinear_grouped_grad_x(res, o, layer.packed, out=new(t, k))
        sbn.bitlinear_grouped_grad_w(res, q, s, o, out=new(2, n_out, k))
        g.check()


@gpu
def test_side_stream_and_graph(sbn_lib, cuda_ok):
    """The calls on another stream than the current one, and captured: two
    graphs that share no buffers replayed together with eager calls."""
    sbn = _sbn()
    k, n_out, n, m = 512, 520, 6, 8
    layer = Layer(4, n_out, k, n, m, "graph")
    for rows in (12, 200):
        x, q, s = acts_of(rows, k, f"graph{rows}")
        o = torch.tensor([0, rows // 4, rows // 2, rows // 2, rows], dtype=torch.int32, device="cuda")
        dy = (1e-2 * torch.randn(rows, n_out, device="cuda")).to(torch.bfloat16)

        def step(stream=None):
            z = torch.empty(rows, n_out, dtype=torch.bfloat16, device="cuda")
            y = sbn.bitlinear_grouped_x(x, o, layer.packed, act="silu", out_z=z, stream=stream)
            d, db = sbn.act_grad(dy, z, "silu", offsets=o, stream=stream)
            return (y, d, db, sbn.bitlinear_grouped_grad_x(d, o, layer.packed, stream=stream),
                    sbn.bitlinear_grouped_grad_w(d, q, s, o, stream=stream),
                    sbn.bitlinear_x_act(x, layer.packed.expert(1), act="gelu", stream=stream))
        want = step()
        clean(sbn)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = step(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs = step()
            graphs.append((g, outs))
        # other routing in the same buffers: the offsets are read at replay
        o.copy_(torch.tensor([0, 1, rows - 2, rows - 1, rows], dtype=torch.int32))
        want = step()
        for g, outs in graphs:
            for t in outs:
                t.zero_()
        for g, _ in graphs:
            g.replay()
        clean(sbn)
        for _, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


@gpu
def test_refusals_of_the_binding(sbn_lib, cuda_ok):
    sbn = _sbn()
    layer = Layer(2, 64, 256, 2, 4, "ref")
    w, we = layer.packed, layer.packed.expert(0)
    x, q, s = acts_of(20, 256, "ref")
    o = torch.tensor([0, 5, 20], dtype=torch.int32, device="cuda")
    y = torch.empty(20, 64, dtype=torch.bfloat16, device="cuda")
    bad = [
        (ValueError, lambda: sbn.bitlinear_act(q, s, we, act="tanh")),
        (ValueError, lambda: sbn.bitlinear_act(q[:, :128].contiguous(), s, we)),
        (ValueError, lambda: sbn.bitlinear_act(q[:, ::2], s, we)),
        (ValueError, lambda: sbn.bitlinear_act(q, s[:5], we)),
        (ValueError, lambda: sbn.bitlinear_act(q, s, we, bias=torch.zeros(63, device="cuda"))),
        (TypeError, lambda: sbn.bitlinear_act(q, s, we, bias=torch.zeros(64, device="cuda", dtype=torch.bfloat16))),
        (ValueError, lambda: sbn.bitlinear_act(q, s, we, residual=y[:10])),
        (ValueError, lambda: sbn.bitlinear_act(q, s, we, out=y, out_z=y)),
        (ValueError, lambda: sbn.bitlinear_act(q, s, we, bias=torch.zeros(64))),
        (sbn.SbnError, lambda: sbn.bitlinear_x_act(x, we, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
        (TypeError, lambda: sbn.bitlinear_grouped(q, s, o.long(), w)),
        (ValueError, lambda: sbn.bitlinear_grouped(q, s, o[:2], w)),
        (ValueError, lambda: sbn.bitlinear_grouped(q, s, o.cpu(), w)),
        (ValueError, lambda: sbn.bitlinear_grouped(q, s, o, w, bias=torch.zeros(64, device="cuda"))),
        (ValueError, lambda: sbn.bitlinear_grouped_grad_x(y[:, :32].contiguous(), o, w)),
        (ValueError, lambda: sbn.bitlinear_grouped_grad_w(y[:5], q, s, o)),
        (ValueError, lambda: sbn.act_grad(y, y[:5], "relu")),
        (ValueError, lambda: sbn.act_grad(y, y, "relu", out=y)),
        (ValueError, lambda: sbn.quantize_experts(layer.latent, 2, 4, out=sbn.alloc_experts(3, 64, 256, 2, 4, "cuda"))),
    ]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            pytest.fail(f"call {i} was not refused")
    clean(sbn)


@gpu
def test_training_step_of_an_expert_block(sbn_lib, cuda_ok):
    """A ternary expert block as it is trained: quantize the latents, up with
    bias and relu2, down, backward through both, AdamW on the fp32 masters,
    whose bf16 copies are quantized again. Every gradient against the same
    chain in float64 on the operands the calls received."""
    sbn = _sbn()
    E, d, f, rows = 4, 256, 384, 150
    sizes = (70, 0, 30, 50)
    off = np.concatenate([[0], np.cumsum(sizes)])
    spans = list(zip(off[:-1].tolist(), off[1:].tolist()))
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    masters = [0.02 * torch.randn(E, f, d, device="cuda", generator=g), 0.02 * torch.randn(E, d, f, device="cuda", generator=g),
               torch.zeros(E, f, device="cuda")]
    latents = [t.to(torch.bfloat16) for t in masters]
    opt = sbn.AdamW(masters, lr=1e-2, copies=latents, state_bits=8, seed=1)
    x = torch.randn(rows, d, device="cuda", generator=g).to(torch.bfloat16)
    dy = (1e-2 * torch.randn(rows, d, device="cuda", generator=g)).to(torch.bfloat16)
    flips = []
    for _ in range(2):
        up, down = sbn.quantize_experts(latents[0], 6, 8), sbn.quantize_experts(latents[1], 6, 8)
        xq, xs = torch.empty(rows, d, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
        z, hq, hs = (torch.empty(rows, f, dtype=torch.bfloat16, device="cuda"),
                     torch.empty(rows, f, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda"))
        h = sbn.bitlinear_grouped_x(x, o, up, bias=masters[2], act="relu2", out_z=z, out_q=xq, out_s=xs)
        sbn.bitlinear_grouped_x(h, o, down, out_q=hq, out_s=hs)
        dw2 = sbn.bitlinear_grouped_grad_w(dy, hq, hs, o)
        dh = sbn.bitlinear_grouped_grad_x(dy, o, down)
        dz, db = sbn.act_grad(dh, z, "relu2", offsets=o)
        dw1 = sbn.bitlinear_grouped_grad_w(dz, xq, xs, o)
        sbn.bitlinear_grouped_grad_x(dz, o, up)
        clean(sbn)
        for e, (a, b) in enumerate(spans):
            for got, dd, qq, ss in ((dw2[e], dy, hq, hs), (dw1[e], dz, xq, xs)):
                xd = qq[a:b].double() * ss[a:b].double()[:, None] / 127
                close(got, *dw_reference(dd[a:b].double(), xd), f"dw {e}")
            ref = dh[a:b].double() * 2 * z[a:b].double().clamp(min=0)
            close(dz[a:b], ref, (H + 4 * U) * ref.abs(), f"dz {e}")
            close(db[e], ref.sum(0), (b - a + 16) * U * ref.abs().sum(0), f"dbias {e}")
        before = masters[0].clone()
        # the optimizer takes gradients of one type: the bias gradient joins in bf16
        opt.step([dw1, dw2, db.to(torch.bfloat16)])
        torch.cuda.synchronize()
        assert not torch.equal(before, masters[0])
        assert all(torch.equal(c, p.to(torch.bfloat16)) for c, p in zip(latents, masters))
        again = sbn.quantize_experts(latents[0], 6, 8)
        flips.append(int(sbn.mask_flips(up.expert(0), again.expert(0))))
    assert all(c > 0 for c in flips)
    clean(sbn)


@gpu
@pytest.mark.parametrize("n_out", [64, 129])
def test_act_grad_offsets_out_of_order(sbn_lib, cuda_ok, n_out):
    """No row belongs to two experts whatever the offsets are: dz in place is
    formed once, and the sums are those of the clamped offsets."""
    sbn = _sbn()
    rows = 300
    g = torch.Generator(device="cuda").manual_seed(5)
    dy = torch.randn(rows, n_out, device="cuda", generator=g).to(torch.bfloat16)
    z = torch.randn(rows, n_out, device="cuda", generator=g).to(torch.bfloat16)
    for bad, good in (([0, 200, 100, 150, 300], [0, 200, 200, 200, 300]), ([-7, 40, -1, 5000, 90], [0, 40, 40, 300, 300]),
                      ([500, 0, 20, 30, 40], [300, 300, 300, 300, 300])):
        want, wsum = sbn.act_grad(dy, z, "silu", torch.tensor(good, dtype=torch.int32, device="cuda"), out=dy.clone())
        d = dy.clone()
        got, gsum = sbn.act_grad(d, z, "silu", torch.tensor(bad, dtype=torch.int32, device="cuda"), out=d)
        clean(sbn)
        assert torch.equal(got, want) and torch.equal(gsum, wsum), bad


@gpu
@pytest.mark.parametrize("t", [3, 40])
def test_nan_and_infinity_pass_through(sbn_lib, cuda_ok, t):
    """A bias that is not finite reaches the output as in the formula: no
    activation hides a NaN."""
    sbn = _sbn()
    layer = Layer(1, 64, 256, 6, 8, "nan")
    x, q, s = acts_of(t, 256, f"nan{t}")
    bias = torch.zeros(64, device="cuda")
    bias[3], bias[5], bias[7] = float("nan"), float("inf"), float("-inf")
    for act, low in (("none", float("-inf")), ("relu", 0.0), ("relu2", 0.0), ("silu", None), ("gelu", None)):
        for y in (sbn.bitlinear_act(q, s, layer.packed.expert(0), bias=bias, act=act),
                  sbn.bitlinear_act(q, s, layer.packed.expert(0), bias=bias, act=act, workspace=False)):
            assert y[:, 3].isnan().all() and (y[:, 5] == float("inf")).all(), act
            if low is not None:
                assert (y[:, 7] == low).all(), act
            assert y[:, [0, 1, 2, 4, 6, 8]].isfinite().all()
    clean(sbn)
