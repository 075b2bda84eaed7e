"""AdamW over many tensors: fp32 states against a 64-bit step, 8-bit states
bit for bit against their definition in numpy fp32, and the argument checks.

Tolerances of the fp32 step, u = 2^-24 (half a step of fp32): b1 m and
(1 - b1) g carry two roundings each (coefficient, product) and the sum one,
so m is within 3 u of M = |b1 m| + |(1 - b1) g|; v likewise within 4 u
(one product more). 6 u and 8 u are asserted. The update a m / (r c2 + eps)
has a: lr / bc1 (expm1f is within 2 steps = 4 u, argument 1 u, division 1 u:
6 u), the root of v (2 + 1 u), c2 (4 u), product and sum (2 u), reciprocal (4 u) and
two products (2 u): 21 u of a M / den in all with m's own 6 u on top; 32 u is
asserted, plus 3 u |p| for the decay's coefficient, product and the last
difference.
"""

import numpy as np
import pytest
import torch

U = 2.0 ** -24
BLOCK = 256


def _sbn():
    from sparse_linear_layers_fwd_b200 import sbn
    return sbn


# --------------------------------------------------------------------------
# numpy definition of the 8-bit states
# --------------------------------------------------------------------------
def np_mix(x):
    x = x.astype(np.uint64) & 0xFFFFFFFF
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0xB7E15163)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def np_uniform(numel, seed, t, tensor):
    key = np_mix(np.array([(seed + t * 0x9E3779B1 + tensor * 0xB7E15163) & 0xFFFFFFFF]))[0]
    h = np_mix(np.arange(numel, dtype=np.uint64) ^ key)
    f = np.float32
    return (h & np.uint64(0xFFFF)).astype(f) * f(2.0 ** -16), (h >> np.uint64(16)).astype(f) * f(2.0 ** -16)


def np_codes(x, u, root):
    """fp32 x -> (values of the e4m3 codes, scales per block)."""
    f = np.float32
    n = x.size
    pad = -n % BLOCK
    xb = np.pad(np.abs(x), (0, pad)).reshape(-1, BLOCK)
    _, e = np.frexp(xb.max(axis=1))
    e = np.where(xb.max(axis=1) > 0, np.maximum(e - 1, -100), -100)
    y = (xb * np.ldexp(f(1), 7 - e).astype(f)[:, None]).reshape(-1)[:n].astype(f)
    _, ey = np.frexp(y)
    ey = np.where(y > 0, np.maximum(ey - 1, -6), -6)
    ulp = np.ldexp(f(1), ey - 3).astype(f)
    s = (y / ulp).astype(f)
    k = np.floor(s)
    up = (u * (k + k + f(1)) < (s - k) * (s + k)) if root else (u < s - k)
    q = ((k + up.astype(f)) * ulp).astype(f)
    if root:
        q = np.where(y > 0, np.maximum(q, f(2.0 ** -9)), q)
    return np.copysign(q, x).astype(f), np.ldexp(f(1), e - 7).astype(f)


def test_rounding_keeps_expectations():
    # the exact expectations of the two rules at points of the grid's interior
    f = np.float32
    for root in (False, True):
        for n in (1, 7, 8, 11, 15):
            s = np.float64(n) + np.linspace(0.01, 0.99, 13)
            p = (s * s - n * n) / (2 * n + 1) if root else s - n
            kept = n ** 2 + p * (2 * n + 1) if root else n + p
            assert np.allclose(kept, s * s if root else s, rtol=1e-14)
    # the hash's halves are uniform and not correlated with each other or along the index
    a, b = np_uniform(1 << 18, 5, 3, 2)
    sd = 1 / np.sqrt(12 * a.size)
    for h in (a, b):
        assert abs(h.mean(dtype=np.float64) - 0.5) < 5 * sd
        assert abs(np.corrcoef(h[:-1], h[1:])[0, 1]) < 5 / np.sqrt(h.size)
    assert abs(np.corrcoef(a, b)[0, 1]) < 5 / np.sqrt(a.size)
    assert f(1) > a.max()


# --------------------------------------------------------------------------
# CPU: the C entry's checks
# --------------------------------------------------------------------------
A = 0x10000


def adamw_call(lib, entries=((A, A, A, A, A, A, 0, 64),), count=None, pb=0, gb=1, bits=32, step=A, lr=1e-3, lrd=None,
               b1=0.9, b2=0.95, eps=1e-5, wd=0.1, gs=None):
    tab = np.array(entries, dtype=np.int64)
    return lib.sbn_adamw(tab.ctypes.data, len(entries) if count is None else count, pb, gb, bits, step, lr, lrd, b1, b2,
                         eps, wd, gs, 0, None)


def test_adamw_validation(sbn_lib):
    lib = sbn_lib
    e = (A, A, A, A, A, A, 0, 64)

    def with_(i, v):
        return (tuple(v if j == i else x for j, x in enumerate(e)),)
    assert lib.sbn_adamw(None, 1, 0, 1, 32, A, 1e-3, None, 0.9, 0.95, 1e-5, 0.1, None, 0, None) == 1
    assert adamw_call(lib, step=None) == 1
    for i in range(4):
        assert adamw_call(lib, with_(i, 0)) == 1
    assert adamw_call(lib, with_(4, 0), bits=8) == 1
    assert adamw_call(lib, with_(5, 0), bits=8) == 1
    assert adamw_call(lib, count=0) == 2
    assert adamw_call(lib, bits=16) == 2
    assert adamw_call(lib, with_(7, -1)) == 2
    assert adamw_call(lib, with_(7, 1 << 31)) == 2
    assert adamw_call(lib, b1=1.0) == 2
    assert adamw_call(lib, b2=-0.1) == 2
    assert adamw_call(lib, eps=-1.0) == 2
    assert adamw_call(lib, eps=0.0) == 2
    assert adamw_call(lib, eps=float("nan")) == 2
    assert adamw_call(lib, lr=float("inf")) == 2
    assert adamw_call(lib, with_(6, A), pb=1) == 2          # no copy of bf16 parameters
    assert adamw_call(lib, with_(0, A + 2)) == 4
    assert adamw_call(lib, with_(1, A + 1)) == 4
    assert adamw_call(lib, with_(2, A + 1)) == 4
    assert adamw_call(lib, step=A + 2) == 4
    assert adamw_call(lib, lrd=A + 1) == 4


def test_adamw_class_refuses_on_cpu(sbn_lib):
    sbn = _sbn()
    with pytest.raises(ValueError):
        sbn.AdamW([])
    with pytest.raises(ValueError):
        sbn.AdamW([torch.zeros(4)])                           # not a CUDA tensor
    with pytest.raises(TypeError):
        sbn.AdamW([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(ValueError):
        sbn.AdamW([torch.zeros(4)], state_bits=16)


# --------------------------------------------------------------------------
# GPU
# --------------------------------------------------------------------------
gpu = pytest.mark.gpu


def _tensors(sizes, dtype, rng, scale, offset=0):
    """One tensor per size; offset > 0 makes it a view that many elements into
    a larger buffer (not aligned for wide accesses). Canaries around."""
    out, bufs = [], []
    for n in sizes:
        buf = torch.full((n + 64 + offset,), 7.0, dtype=dtype, device="cuda")
        v = buf[32 + offset:32 + offset + n]
        v.copy_(torch.from_numpy(rng.standard_normal(n) * scale).to(dtype))
        out.append(v)
        bufs.append((buf, 32 + offset, n))
    return out, bufs


def _edges_intact(bufs):
    for buf, a, n in bufs:
        b = buf.float()
        assert (b[:a] == 7.0).all() and (b[a + n:] == 7.0).all()


SIZES = [1, 7, 8, 255, 256, 257, 2048, 2049, 0, 5000, 100003]


def _np(t):
    return t.detach().float().cpu().numpy()


@gpu
@pytest.mark.parametrize("pdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_fp32_states(sbn_lib, cuda_ok, pdt, gdt, offset):
    sbn = _sbn()
    rng = np.random.default_rng(1)
    p, pb = _tensors(SIZES, pdt, rng, 0.02, offset)
    copies, cb = _tensors(SIZES, torch.bfloat16, rng, 1.0, offset) if pdt == torch.float32 else (None, [])
    lr, b1, b2, eps, wd = 3e-3, 0.9, 0.95, 1e-8, 0.1
    opt = sbn.AdamW(p, lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd, copies=copies)
    scale = torch.tensor([0.5], device="cuda")
    for t in range(1, 4):
        g, _ = _tensors(SIZES, gdt, rng, 1e-3, offset)
        before = [(_np(a).astype(np.float64), _np(b).astype(np.float64), _np(c).astype(np.float64))
                  for a, b, c in zip(opt.params, opt.m, opt.v)]
        opt.step(g, grad_scale=scale)
        torch.cuda.synchronize()
        assert opt.step_state.tolist() == [t, 0]
        for i, (p0, m0, v0) in enumerate(before):
            gd = _np(g[i]).astype(np.float64) * 0.5
            m = b1 * m0 + (1 - b1) * gd
            v = b2 * v0 + (1 - b2) * gd * gd
            mabs = b1 * np.abs(m0) + (1 - b1) * np.abs(gd)
            a, den = lr / (1 - b1 ** t), np.sqrt(v / (1 - b2 ** t)) + eps
            ref = p0 * (1 - lr * wd) - a * m / den
            assert (np.abs(_np(opt.m[i]) - m) <= 6 * U * mabs + 1e-45).all()
            assert (np.abs(_np(opt.v[i]) - v) <= 8 * U * v + 1e-45).all()
            tol = 3 * U * np.abs(p0) + 32 * U * a * mabs / den
            if pdt == torch.bfloat16:
                tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
            assert (np.abs(_np(p[i]) - ref) <= tol).all(), i
            if copies is not None:   # the rounded master, exactly
                assert torch.equal(copies[i], p[i].to(torch.bfloat16))
    _edges_intact(pb + cb)


@gpu
@pytest.mark.parametrize("pdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 3])
def test_8bit_states_bit_for_bit(sbn_lib, cuda_ok, pdt, offset):
    sbn = _sbn()
    f = np.float32
    rng = np.random.default_rng(2)
    p, pb = _tensors(SIZES, pdt, rng, 0.02, offset)
    lr, b1, b2, eps, wd, seed = 1e-3, 0.9, 0.999, 1e-8, 0.01, 0xFFFFFFF0
    opt = sbn.AdamW(p, lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd, state_bits=8, seed=seed)
    if offset:   # states at odd addresses
        opt.m = [torch.zeros(n + offset, dtype=torch.float8_e4m3fn, device="cuda")[offset:] for n in SIZES]
        opt.v = [torch.zeros(n + offset, dtype=torch.float8_e4m3fn, device="cuda")[offset:] for n in SIZES]
    for t in range(1, 5):
        g, _ = _tensors(SIZES, torch.bfloat16, rng, 1e-3, offset)
        for x in g:   # a wide range inside each block, zeros among it
            x.mul_(torch.exp2(torch.randint(-14, 3, x.shape, device="cuda").float()).to(x.dtype))
            x[::5] = 0
        old = [(_np(a), _np(b), _np(c), _np(d), _np(e)) for a, b, c, d, e in
               zip(p, opt.m, opt.v, opt.m_scales, opt.v_scales)]
        opt.step(g)
        torch.cuda.synchronize()
        for i, (p0, mc, vc, ms, vs) in enumerate(old):
            n = SIZES[i]
            gi = _np(g[i])
            rep = lambda s: np.repeat(s, BLOCK)[:n]  # noqa: E731
            m = (f(b1) * (mc * rep(ms)) + f(1 - b1) * gi).astype(f)
            r0 = vc * rep(vs)
            v = (f(b2) * (r0 * r0) + f(1 - b2) * (gi * gi)).astype(f)
            r = np.sqrt(v)
            um, ur = np_uniform(n, seed, t, i)
            if n == 0:
                continue
            for x, u, root, got, sc in ((m, um, False, opt.m[i], opt.m_scales[i]), (r, ur, True, opt.v[i], opt.v_scales[i])):
                q, s = np_codes(x, u, root)
                assert np.array_equal(_np(sc), s), (t, i)
                assert np.array_equal(_np(got), q), (t, i, np.flatnonzero(_np(got) != q)[:5])
            # the parameters move by the averages before they are rounded
            a = lr / (1 - b1 ** t)
            den = r.astype(np.float64) / np.sqrt(1 - b2 ** t) + eps
            ref = p0.astype(np.float64) * (1 - lr * wd) - a * m.astype(np.float64) / den
            tol = 3 * U * np.abs(p0) + 32 * U * a * np.abs(m) / den
            if pdt == torch.bfloat16:
                tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
            assert (np.abs(_np(p[i]) - ref) <= tol).all()
    _edges_intact(pb)


@gpu
def test_8bit_averages_follow_the_exact_ones(sbn_lib, cuda_ok):
    """With a constant gradient v rises from 0 to g^2 like 1 - b2^t, whatever
    the codes' width: the rounding keeps the expectation. 65536 elements,
    300 steps of b2 = 0.99. A step's rounding noise in v is at most
    d (1 - d) of the code's width squared; per element the stationary spread
    stays below 0.5 g^2, so the mean of 65536 is within 5 * 0.5 / 256 < 1%."""
    sbn = _sbn()
    n, g0 = 65536, 2.0 ** -7 * 1.3
    p = torch.zeros(n, device="cuda")
    opt = sbn.AdamW([p], lr=0.0, betas=(0.9, 0.99), weight_decay=0.0, state_bits=8, seed=11)
    g = torch.full((n,), g0, device="cuda")
    for _ in range(300):
        opt.step([g])
    r = opt.v[0].float().view(-1, BLOCK) * opt.v_scales[0][:, None]
    m = opt.m[0].float().view(-1, BLOCK) * opt.m_scales[0][:, None]
    v_mean = (r.double() ** 2).mean().item()
    want = g0 * g0 * (1 - 0.99 ** 300)
    assert abs(v_mean / want - 1) < 0.01
    assert abs(m.double().mean().item() / g0 - 1) < 0.01


@gpu
def test_many_tensors_and_graph_replay(sbn_lib, cuda_ok):
    """More tensors than one launch's table, captured and replayed with a
    learning rate read from the device: the same as eager steps."""
    sbn = _sbn()
    sizes = [1 + (37 * i) % 700 for i in range(1000)]
    for bits in (32, 8):
        runs = []
        for graph in (False, True):
            rng = np.random.default_rng(3)
            p, _ = _tensors(sizes, torch.float32, rng, 0.02)
            g, _ = _tensors(sizes, torch.bfloat16, rng, 1e-3)
            lr = torch.tensor([1e-3], device="cuda")
            opt = sbn.AdamW(p, lr=lr, state_bits=bits, seed=4)
            opt.step(g)
            if graph:
                torch.cuda.synchronize()
                cg = torch.cuda.CUDAGraph()
                with torch.cuda.graph(cg):
                    opt.step(g)
            for k in range(3):
                lr.fill_(1e-3 / (k + 1))
                cg.replay() if graph else opt.step(g)
            torch.cuda.synchronize()
            assert opt.step_state.tolist() == [4, 0]
            runs.append([t.float().cpu() for ts in (p, opt.m, opt.v) for t in ts])
        assert all(torch.equal(a, b) for a, b in zip(*runs)), bits


@gpu
def test_state_dict_streams_and_refusals(sbn_lib, cuda_ok):
    sbn = _sbn()
    rng = np.random.default_rng(5)
    sizes = [300, 4096]
    p, _ = _tensors(sizes, torch.float32, rng, 0.02)
    g, _ = _tensors(sizes, torch.float32, rng, 1e-3)
    opt = sbn.AdamW(p, state_bits=8, seed=9)
    opt.step(g)
    saved, p_saved = opt.state_dict(), [x.clone() for x in p]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    opt.step(g, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    first = [x.clone() for x in p]
    other = sbn.AdamW(p_saved, state_bits=8, seed=9)
    other.load_state_dict(saved)
    other.step(g)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, p_saved))
    with pytest.raises(ValueError):
        opt.step(g[:1])
    with pytest.raises(ValueError):
        opt.step([g[1], g[0]])
    with pytest.raises(TypeError):
        opt.step([x.half() for x in g])
    with pytest.raises(TypeError):
        opt.step([g[0], g[1].to(torch.bfloat16)])
    with pytest.raises(ValueError):
        sbn.AdamW([p[0], p[0]])
    with pytest.raises(TypeError):
        sbn.AdamW([x.to(torch.bfloat16) for x in p], copies=p)
    with pytest.raises(ValueError):
        sbn.AdamW([torch.zeros(8, 8, device="cuda").t()[:, :4]])
    with pytest.raises(ValueError):
        other.load_state_dict(sbn.AdamW(p).state_dict())


@gpu
def test_overlaps_and_exchanged_storage(sbn_lib, cuda_ok):
    sbn = _sbn()
    flat = torch.randn(1000, device="cuda")
    for parts in ([flat[:600], flat[599:]], [flat, flat], [flat[:10], flat[20:30], flat[25:40]]):
        with pytest.raises(ValueError):
            sbn.AdamW(parts)
    with pytest.raises(ValueError):
        sbn.AdamW([flat], copies=[flat.view(torch.bfloat16)[:1000]])
    opt = sbn.AdamW([flat[:600], flat[600:]], lr=0.1, weight_decay=0.0)   # neighbours are apart
    grads = [torch.ones(600, device="cuda"), torch.ones(400, device="cuda")]
    before = flat.clone()
    opt.step(grads)
    torch.cuda.synchronize()
    assert bool((flat < before).all())
    # storage exchanged for one of the same kind is followed, any other refused
    p = torch.zeros(64, 8, device="cuda")
    opt = sbn.AdamW([p], lr=0.1, weight_decay=0.0)
    p.data = torch.ones(64, 8, device="cuda")
    g = [torch.ones(64, 8, device="cuda")]
    opt.step(g)
    torch.cuda.synchronize()
    assert bool((p < 1).all())
    for other in (torch.ones(32, 8, device="cuda"), torch.ones(8, 64, device="cuda").t(),
                  torch.ones(64, 8, device="cuda", dtype=torch.bfloat16), torch.ones(64, 8)):
        p.data = other
        with pytest.raises(ValueError):
            opt.step(g)
    assert int(opt.step_state[0]) == 1 and sbn.get_device_error() == 0
