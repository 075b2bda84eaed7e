"""The feed-forward calls where they can go wrong beside the sizes of
test_feedforward.py, whose references and tolerances serve here too."""

import numpy as np
import pytest
import torch

from test_feedforward import H, U, acts_of, clean, close, dw_reference, epilogue_inputs, reference

gpu = pytest.mark.gpu

SMEM = 227 * 1024    # shared memory of a CTA


def _sbn():
    from sparse_linear_layers_fwd_b200 import sbn
    return sbn


class Repeated:
    """`experts` experts that share the weights of a few layers: expert e has
    those of layer e modulo their number."""

    def __init__(self, few, experts):
        sbn = _sbn()
        p, pick = few.packed, torch.arange(experts, device="cuda") % few.packed.experts
        self.packed = sbn.PackedExperts(p.codes[pick], None if p.meta is None else p.meta[pick], p.gamma[pick], p.n_out, p.k,
                                        p.n, p.m, experts)
        self.gamma = few.gamma[pick]

        class Dense(list):
            shape = (experts, p.n_out, p.k)
        self.dense = Dense(few.dense[i] for i in pick.tolist())


class Packed:
    """Experts quantized on the device, their ternary matrices read back from
    the packed arrays (the quantizer's own parity tests pin those)."""

    def __init__(self, experts, n_out, k, n, m, tag):
        sbn = _sbn()
        g = torch.Generator(device="cuda").manual_seed(len(tag) + n_out + k)
        w = (0.02 * torch.randn(experts, n_out, k, device="cuda", generator=g)).to(torch.bfloat16)
        self.packed = p = sbn.quantize_experts(w, n, m)
        kept = n_out * (k * n // m)
        two = torch.tensor([0, 2, 4, 6], device="cuda")
        bit = torch.arange(8, device="cuda")
        value = torch.tensor([0, 1, 0, -1], dtype=torch.int8, device="cuda")
        self.dense = []
        for e in range(experts):
            codes = value[((p.codes[e][..., None] >> two) & 3).long()].view(n_out, -1)[:, :k * n // m]
            if n == m:
                self.dense.append(codes.double())
                continue
            keep = ((p.meta[e][..., None] >> bit) & 1).bool().view(n_out, -1)[:, :k]
            assert int(keep.sum()) == kept
            d = torch.zeros(n_out, k, dtype=torch.float64, device="cuda")
            d[keep] = codes.reshape(-1).double()
            self.dense.append(d)
        self.gamma = p.gamma.double()

        class Dense(list):
            shape = (experts, n_out, k)
        self.dense = Dense(self.dense)


# rows per expert, K, N_out, pattern: one to three items of 256 positions to a
# tile and 17 to 56 tiles to a CTA, 8 and 16 rows, one layer and experts; and rows
# so long that shared memory leaves a CTA fewer slots than it has tiles
RING_CASES = [
    ((1,) * 16, 128, 8000, 6, 8),
    ((1,) * 16, 256, 8192, 2, 4),
    ((1,) * 8, 256, 5057, 6, 8),
    ((1,) * 8, 512, 8000, 8, 8),
    ((2, 0, 1, 1) * 4, 512, 5000, 8, 16),
    ((1,) * 12, 768, 4000, 4, 8),
    ((1,), 256, 50304, 6, 8),
    ((7,), 128, 60001, 1, 4),
    ((1,), 8192, 19000, 6, 8),
    ((2, 2), 4096, 19000, 12, 16),
]


@gpu
@pytest.mark.parametrize("case", RING_CASES, ids=[f"e{len(c[0])}_r{sum(c[0])}_k{c[1]}_n{c[2]}_{c[3]}of{c[4]}" for c in RING_CASES])
def test_decode_ring_reused(sbn_lib, cuda_ok, case):
    """At most 16 rows whose CTAs walk more 16-feature tiles than their ring of
    shared memory has slots: every slot is waited for, filled and handed back
    several times. INT8 and bf16 activations, the same bits on every run."""
    sbn = _sbn()
    sizes, k, n_out, n, m = case
    rows, experts = sum(sizes), len(sizes)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    active = sum(1 for s in sizes if s)
    least = active * ((n_out + 15) // 16) // sms
    slots = min(16, SMEM // (16 * (sbn.codes_row_bytes(k, n, m) + sbn.meta_row_bytes(k, n, m))))
    assert least > slots, "every CTA must have more tiles than slots"
    layer = Packed(experts, n_out, k, n, m, "ring")
    off = np.concatenate([[0], np.cumsum(sizes)])
    spans = list(zip(off[:-1].tolist(), off[1:].tolist()))
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    x, q, s = acts_of(rows, k, f"ring{case}"[:40])
    bias, res = epilogue_inputs(rows, n_out, experts)
    y, ytol, z, ztol = reference(layer, q, s, spans, bias, "silu", res)
    tiny = torch.empty(16, dtype=torch.uint8, device="cuda")   # too small for any other route
    first = None
    for turn in range(6):
        out = torch.full((rows, n_out), 77.0, dtype=torch.bfloat16, device="cuda")
        oz = torch.full_like(out, 78.0)
        if turn % 2:
            sbn.bitlinear_grouped(q, s, o, layer.packed, bias=bias, act="silu", residual=res, out=out, out_z=oz)
        else:
            sbn.bitlinear_grouped_x(x, o, layer.packed, bias=bias, act="silu", residual=res, out=out, out_z=oz,
                                    workspace=tiny)
        clean(sbn)
        close(out, y, ytol, f"y {turn}")
        close(oz, z, ztol, f"z {turn}")
        if first is None:
            first = (out, oz)
        assert torch.equal(out, first[0]) and torch.equal(oz, first[1])
    if experts == 1:
        w = layer.packed.expert(0)
        for out in (sbn.bitlinear_x_act(x, w, bias=bias[0], act="silu", residual=res, workspace=tiny),
                    sbn.bitlinear_act(q, s, w, bias=bias[0], act="silu", residual=res)):
            assert torch.equal(out, first[0])
    clean(sbn)


@gpu
@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 700])
def test_act_grad_at_the_last_rows(sbn_lib, cuda_ok, rows):
    """One feature and as many rows as a call may have: the rows behind the
    last are counted, not wrapped around. Only the last 3000 belong to a group,
    the very last to one of its own; dz and the sums are small whole numbers."""
    sbn = _sbn()
    n = 3000
    dy = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda")
    z = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda")
    dy[:2 * n] = 5.0
    dy[-2 * n:] = 5.0
    v = torch.arange(n, device="cuda") % 7 - 3
    dy[-n:, 0] = v.to(torch.bfloat16)
    z[-n:] = 1.0
    o = torch.tensor([rows - n, rows - 1, rows], dtype=torch.int32, device="cuda")
    _, db = sbn.act_grad(dy, z, "relu2", offsets=o, out=dy)
    clean(sbn)
    assert torch.equal(dy[-n:, 0], (2 * v).to(torch.bfloat16))
    assert bool((dy[-2 * n:-n] == 5.0).all()) and bool((dy[:2 * n] == 5.0).all())
    assert db.view(-1).tolist() == [float(2 * v[:-1].sum()), float(2 * v[-1])]


@gpu
@pytest.mark.parametrize("limit_ns", [1000, 200_000])
def test_a_warp_gives_up_as_one(sbn_lib, cuda_ok, limit_ns):
    """Half a warp waits for a barrier that never comes, half for one that has:
    no lane may be told that the wait went well (it would clear the error)."""
    sbn = _sbn()
    clean(sbn)
    for _ in range(20):
        sbn.selftest_wait_timeout(0, limit_ns)
        torch.cuda.synchronize()
        assert sbn.SBN_STATUS[sbn.get_device_error()] == "SBN_ERR_TIMEOUT"
    clean(sbn)


@gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_keeps_what_is_not_finite(sbn_lib, cuda_ok, bits):
    """NaN and infinite gradients: p, m and v of these elements are not finite
    afterwards (8 bits: the NaN code) and stay so; all others and the scales are
    those of a run in which they were zero, bit for bit."""
    sbn = _sbn()
    n = 1000
    g = torch.Generator(device="cuda").manual_seed(6)
    p0 = 0.02 * torch.randn(n, device="cuda", generator=g)
    g0 = 1e-3 * torch.randn(n, device="cuda", generator=g)
    bad = {0: float("nan"), 7: float("inf"), 200: float("-inf"), 255: float("nan"), 300: float("inf"), 999: float("nan")}
    at = torch.tensor(sorted(bad), device="cuda")
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[at] = False
    g0[at] = 0.0
    runs = []
    for broken in (False, True):
        p, grad = p0.clone(), g0.clone()
        if broken:
            grad[at] = torch.tensor([bad[i] for i in sorted(bad)], device="cuda")
        opt = sbn.AdamW([p], state_bits=bits, seed=3)
        opt.step([grad])
        opt.step([g0])
        clean(sbn)
        runs.append([p, opt.m[0].float(), opt.v[0].float()] + ([opt.m_scales[0], opt.v_scales[0]] if bits == 8 else []))
    for a, b in zip(*(r[:3] for r in runs)):
        assert torch.equal(a[rest], b[rest])
        assert not b[at].isfinite().any()
    assert all(torch.equal(a, b) for a, b in zip(*(r[3:] for r in runs)))
    if bits == 8:
        assert runs[1][1][at].isnan().all() and runs[1][2][at].isnan().all()


@gpu
def test_adamw_checks_its_step_state(sbn_lib, cuda_ok):
    sbn = _sbn()
    p, g = torch.ones(300, device="cuda"), [torch.ones(300, device="cuda")]
    opt = sbn.AdamW([p])
    for err, other in ((ValueError, torch.zeros(2, dtype=torch.int32)), (TypeError, torch.zeros(2, dtype=torch.int64, device="cuda")),
                       (ValueError, torch.zeros(1, dtype=torch.int32, device="cuda")),
                       (ValueError, torch.zeros(4, dtype=torch.int32, device="cuda")[::2])):
        with pytest.raises(err):
            opt.step_state = other
    opt.step_state = mine = torch.tensor([41, 0], dtype=torch.int32, device="cuda")
    opt.step(g)
    clean(sbn)
    assert mine.tolist() == [42, 0] and opt.state_dict()["step"].tolist() == [42, 0]


@gpu
@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("nm", [(6, 8), (2, 4)])
def test_no_rows(sbn_lib, cuda_ok, nm, side):
    """A batch without rows runs through a whole block and its backward: empty
    outputs, and zeros where the sums run over no rows; the checks stay."""
    sbn = _sbn()
    n, m = nm
    E, d, f = 3, 256, 129
    g = torch.Generator(device="cuda").manual_seed(1)
    up = sbn.quantize_experts((0.02 * torch.randn(E, f, d, device="cuda", generator=g)).to(torch.bfloat16), n, m)
    x = torch.empty(0, d, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream() if side else None
    new = lambda c, dt: torch.empty(0, c, dtype=dt, device="cuda")  # noqa: E731
    z, dy, bias = new(f, torch.bfloat16), new(f, torch.bfloat16), torch.zeros(E, f, device="cuda")
    q, s = sbn.quantize_acts(x, stream=stream)
    assert q.shape == (0, d) and s.shape == (0,)
    kw = dict(act="gelu", residual=new(f, torch.bfloat16), out_z=z, stream=stream)
    ys = [sbn.bitlinear_grouped(q, s, o, up, bias=bias, **kw), sbn.bitlinear_grouped_x(x, o, up, bias=bias, **kw),
          sbn.bitlinear_act(q, s, up.expert(0), bias=bias[0], **kw), sbn.bitlinear_x_act(x, up.expert(0), bias=bias[0], **kw)]
    assert all(y.shape == (0, f) and y.dtype == torch.bfloat16 for y in ys)
    db, dw = torch.full((E, f), 3.0, device="cuda"), torch.full((E, f, d), 3.0, device="cuda").to(torch.bfloat16)
    torch.cuda.synchronize()
    dz, sums = sbn.act_grad(dy, z, "gelu", offsets=o, out_bias=db, stream=stream)
    _, plain = sbn.act_grad(dy, z, "gelu", stream=stream)
    _, none = sbn.act_grad(dy, z, "gelu", out_bias=False, stream=stream)
    dx = sbn.bitlinear_grouped_grad_x(dz, o, up, stream=stream)
    assert sbn.bitlinear_grouped_grad_w(dz, q, s, o, out=dw, stream=stream) is dw
    fresh = sbn.bitlinear_grouped_grad_w(dz, q, s, o, stream=stream)
    clean(sbn)
    assert dz.shape == (0, f) and dx.shape == (0, d) and sums is db and none is None and plain.shape == (f,)
    assert not db.any() and not plain.any() and not dw.any() and not fresh.any() and fresh.shape == (E, f, d)
    with pytest.raises(ValueError):
        sbn.bitlinear_grouped(q, s, o[:2], up)
    with pytest.raises(ValueError):
        sbn.bitlinear_grouped_grad_w(dz, q, s, o, out=dw[:1])


@gpu
def test_packed_arrays_of_other_sizes_are_refused(sbn_lib, cuda_ok):
    """A handle whose arrays do not belong to the sizes beside them would be
    read out of range, a set of experts in a layer's place as its first."""
    from dataclasses import replace
    sbn = _sbn()
    layer = Packed(3, 64, 256, 6, 8, "sizes")
    we, w = layer.packed, layer.packed.expert(0)
    x, q, s = acts_of(20, 256, "sizes")
    o = torch.tensor([0, 5, 5, 20], dtype=torch.int32, device="cuda")
    dy = torch.zeros(20, 64, dtype=torch.bfloat16, device="cuda")
    single = [lambda h: sbn.bitlinear_act(q, s, h), lambda h: sbn.bitlinear_x_act(x, h)]
    grouped = [lambda h: sbn.bitlinear_grouped(q, s, o, h), lambda h: sbn.bitlinear_grouped_x(x, o, h),
               lambda h: sbn.bitlinear_grouped_grad_x(dy, o, h)]
    for calls, good, others in ((single, w, [we]), (grouped, we, [replace(we, gamma=w.gamma)])):
        half = good.codes.flatten()[:good.codes.numel() // 2]
        others += [replace(good, codes=half), replace(good, meta=good.meta.flatten()[16:]), replace(good, n=4),
                   replace(good, gamma=good.gamma.to(torch.bfloat16))]
        for call in calls:
            call(good)
            for h in others:
                with pytest.raises(ValueError):
                    call(h)
            with pytest.raises(sbn.SbnError):
                call(replace(good, meta=None))
    clean(sbn)


@gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_states_take_one_fill_a_kind(sbn_lib, cuda_ok, bits):
    """A new optimizer fills one buffer for each kind of state, whatever the
    number of tensors; its parts are apart and aligned for the wide accesses,
    and a step gives what states of their own give."""
    sbn = _sbn()
    sizes = [1, 256, 0, 257, 5000, 7]
    g = torch.Generator(device="cuda").manual_seed(2)
    p = [torch.randn(n, device="cuda", generator=g) for n in sizes]
    grads = [torch.randn(n, device="cuda", generator=g) for n in sizes]
    one, own = sbn.AdamW([x.clone() for x in p], state_bits=bits), sbn.AdamW([x.clone() for x in p], state_bits=bits)
    kinds = [one.m, one.v] + ([one.m_scales, one.v_scales] if bits == 8 else [])
    assert len({t.untyped_storage().data_ptr() for kind in kinds for t in kind if t.numel()}) == len(kinds)
    spans = sorted((t.data_ptr(), t.data_ptr() + t.nbytes) for kind in kinds for t in kind if t.numel())
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:])) and all(a % 32 == 0 for a, _ in spans)
    assert not any(t.float().any() for t in one.m + one.v) and all((t == 1).all() for kind in kinds[2:] for t in kind)
    own.m, own.v = [t.clone() for t in own.m], [t.clone() for t in own.v]
    if bits == 8:
        own.m_scales, own.v_scales = [t.clone() for t in own.m_scales], [t.clone() for t in own.v_scales]
    for opt in (one, own):
        opt.step(grads)
        opt.step(grads)
    clean(sbn)
    for a, b in ((one.params, own.params), (one.m, own.m), (one.v, own.v)):
        assert all(torch.equal(x.float(), y.float()) for x, y in zip(a, b))


@gpu
@pytest.mark.parametrize("k,n_out,n,m,sizes,tail", [
    (384, 257, 6, 8, (70, 0, 1, 64, 65), 3), (256, 136, 2, 4, (5, 0, 0, 3), 0), (640, 1000, 8, 16, (129, 300), 7), (128, 9, 8, 8, (1,), 0)])
def test_canaries_of_gradient_workspaces(sbn_lib, cuda_ok, k, n_out, n, m, sizes, tail):
    """Workspaces of exactly the reported size, with known bytes on both sides:
    dX's pitched copy of dY, dW's three arrays, the expanded weights; and the
    outputs of act_grad."""
    from test_canaries import Guarded
    sbn = _sbn()
    E, rows = len(sizes), sum(sizes) + tail
    layer = Packed(E, n_out, k, n, m, "guard")
    x, q, s = acts_of(rows, k, f"guard{k}")
    o = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    dy = torch.randn(rows, n_out, device="cuda", generator=g).to(torch.bfloat16)
    z = torch.randn(rows, n_out, device="cuda", generator=g).to(torch.bfloat16)
    gd = Guarded()
    need_x = int(sbn.lib().sbn_bitlinear_grouped_grad_x_workspace_bytes(rows, n_out))
    need_w = int(sbn.lib().sbn_bitlinear_grouped_grad_w2_workspace_bytes(rows, E, k, n_out))
    need_w1 = int(sbn.lib().sbn_bitlinear_grouped_grad_w_workspace_bytes(rows, E, k, n_out))
    assert (need_x > 0) == (n_out % 8 != 0) and need_w > need_w1 > 0
    dx, dw = gd.tensor((rows, k), torch.bfloat16), gd.tensor((E, n_out, k), torch.bfloat16)
    sbn.bitlinear_grouped_grad_x(dy, o, layer.packed, out=dx, workspace=gd.tensor((need_x,), torch.uint8) if need_x else None)
    sbn.bitlinear_grouped_grad_w(dy, q, s, o, out=dw, workspace=gd.tensor((need_w,), torch.uint8))
    sbn.bitlinear_grouped_grad_w(dy, q, s, o, out=gd.tensor((E, n_out, k), torch.bfloat16), workspace=gd.tensor((need_w1,), torch.uint8))
    need = sbn.bitlinear_workspace_bytes(rows, k, n_out)
    sbn.bitlinear_act(q, s, layer.packed.expert(0), act="silu", residual=dy, out=gd.tensor((rows, n_out), torch.bfloat16),
                      out_z=gd.tensor((rows, n_out), torch.bfloat16), workspace=gd.tensor((need,), torch.uint8) if need else None)
    sbn.act_grad(dy, z, "gelu", offsets=o, out=gd.tensor((rows, n_out), torch.bfloat16), out_bias=gd.tensor((E, n_out), torch.float32))
    gd.check()
    inside = slice(0, rows - tail)
    assert torch.equal(dx[inside], sbn.bitlinear_grouped_grad_x(dy, o, layer.packed)[inside])
    assert torch.equal(dw, sbn.bitlinear_grouped_grad_w(dy, q, s, o))
    clean(sbn)


@gpu
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("sizes", [(1, 255, 257, 5000, 8), (3,) * 30])
def test_canaries_of_adamw(sbn_lib, cuda_ok, bits, sizes):
    """Parameters, bf16 copies, states and scales with known bytes around each."""
    from test_canaries import Guarded
    sbn = _sbn()
    gd = Guarded()
    state = torch.float32 if bits == 32 else torch.float8_e4m3fn

    def zeros(n, dtype):
        t = gd.tensor((n,), dtype)
        t.view(torch.uint8).zero_()
        return t
    p, c = [zeros(n, torch.float32) for n in sizes], [zeros(n, torch.bfloat16) for n in sizes]
    opt = sbn.AdamW(p, copies=c, state_bits=bits)
    opt.m, opt.v = [zeros(n, state) for n in sizes], [zeros(n, state) for n in sizes]
    if bits == 8:
        opt.m_scales = [zeros(-(-n // 256), torch.float32) for n in sizes]
        opt.v_scales = [zeros(-(-n // 256), torch.float32) for n in sizes]
    opt.step_state = zeros(2, torch.int32)
    grads = [torch.ones(n, device="cuda") for n in sizes]
    opt.step(grads)
    opt.step(grads)
    gd.check()
    assert all(bool((t < 0).all()) for t in p + c) and opt.step_state.tolist() == [2, 0]


@gpu
@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
def test_adamw_averages_bit_for_bit(sbn_lib, cuda_ok, gdt):
    """32-bit m and v are the products and sums of the formula, each rounded on
    its own in fp32 (numpy does the same); the parameters' quotient goes through
    an approximate reciprocal and has no such property."""
    sbn = _sbn()
    f = np.float32
    n, b1, b2 = 70001, 0.9, 0.95
    g = torch.Generator(device="cuda").manual_seed(9)
    p = torch.randn(n, device="cuda", generator=g)
    opt = sbn.AdamW([p], lr=1e-3, betas=(b1, b2))
    scale = torch.tensor([0.37], device="cuda")
    m, v = np.zeros(n, f), np.zeros(n, f)
    for _ in range(4):
        grad = (torch.randn(n, device="cuda", generator=g) * torch.exp2(torch.randint(-30, 10, (n,), device="cuda").float())).to(gdt)
        opt.step([grad], grad_scale=scale)
        clean(sbn)
        x = grad.float().cpu().numpy() * f(0.37)
        m = f(b1) * m + f(1 - b1) * x
        v = f(b2) * v + f(1 - b2) * (x * x)
        assert m.dtype == f and v.dtype == f
        assert np.array_equal(opt.m[0].cpu().numpy(), m) and np.array_equal(opt.v[0].cpu().numpy(), v)


@gpu
def test_quantize_experts_checks_what_it_writes(sbn_lib, cuda_ok):
    from dataclasses import replace
    sbn = _sbn()
    w = torch.randn(3, 64, 256, device="cuda").to(torch.bfloat16)
    out = sbn.alloc_experts(3, 64, 256, 6, 8, "cuda")
    for bad in (replace(out, codes=out.codes[:2]), replace(out, meta=out.meta[:2]), replace(out, gamma=out.gamma[:1]),
                replace(out, codes=torch.empty(3, 64, 2 * out.codes.shape[2], dtype=torch.uint8, device="cuda")[..., ::2]),
                replace(out, gamma=out.gamma.cpu())):
        with pytest.raises(ValueError):
            sbn.quantize_experts(w, 6, 8, out=bad)
    with pytest.raises(TypeError):
        sbn.quantize_experts(w, 6, 8, out=out, workspace=torch.empty(1 << 16, device="cuda"))
    with pytest.raises(ValueError):
        sbn.quantize_experts(w, 6, 8, out=out, workspace=torch.empty(1 << 18, dtype=torch.uint8))
    assert sbn.quantize_experts(w, 6, 8, out=out) is out
    again = sbn.quantize_experts(w, 6, 8)
    clean(sbn)
    assert all(torch.equal(a, b) for a, b in ((out.codes, again.codes), (out.meta, again.meta), (out.gamma, again.gamma)))


def run_spans(sizes):
    off = np.concatenate([[0], np.cumsum(sizes)])
    return torch.tensor(off, dtype=torch.int32, device="cuda"), list(zip(off[:-1].tolist(), off[1:].tolist()))


@gpu
@pytest.mark.parametrize("k,n_out", [(128, 1416), (1280, 24)])
def test_more_tiles_than_a_list_holds(sbn_lib, cuda_ok, k, n_out):
    """1000 experts of one or two rows: a CTA of the forward (K = 128) or of dX
    (K = 1280) has more tiles than its list of 64 or 32 worked out ahead."""
    sbn = _sbn()
    E = 1000
    sizes = [1 + e % 2 for e in range(E)]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert E * ((n_out + 127) // 128) // sms > 64 or E * ((k + 255) // 256) // sms > 32
    layer = Repeated(Packed(3, n_out, k, 6, 8, "list"), E)
    o, spans = run_spans(sizes)
    rows = sum(sizes)
    x, q, s = acts_of(rows, k, f"list{k}")
    bias, res = epilogue_inputs(rows, n_out, E)
    y, ytol, z, ztol = reference(layer, q, s, spans, bias, "gelu", res)
    oz = torch.empty(rows, n_out, dtype=torch.bfloat16, device="cuda")
    close(sbn.bitlinear_grouped(q, s, o, layer.packed, bias=bias, act="gelu", residual=res, out_z=oz), y, ytol, "y")
    close(oz, z, ztol, "z")
    dy = res
    dx, dw = sbn.bitlinear_grouped_grad_x(dy, o, layer.packed), sbn.bitlinear_grouped_grad_w(dy, q, s, o)
    clean(sbn)
    xd = q.double() * s.double()[:, None] / 127
    for e, (a, b) in enumerate(spans):
        d, wd = dy[a:b].double(), layer.dense[e] * layer.gamma[e]
        ref, mag = d @ wd, d.abs() @ wd.abs()
        close(dx[a:b], ref, H * ref.abs() + (1 + H) * (2 * n_out + 4) * U * mag, f"dx {e}")
        close(dw[e], *dw_reference(d, xd[a:b]), f"dw {e}")


@gpu
@pytest.mark.parametrize("rows", [12, 400])
def test_weights_past_32_bits(sbn_lib, cuda_ok, rows):
    """300 experts of 2048 x 4096: 2.5e9 weights, so the last experts' dW lies
    past 2^32 bytes and 2^31 elements. Rows in the first, one in the middle and the
    last two experts; the others' dW are zeros."""
    sbn = _sbn()
    E, n_out, k = 300, 2048, 4096
    layer = Repeated(Packed(2, n_out, k, 6, 8, "far"), E)
    sizes = [0] * E
    for e, part in ((0, 1), (171, 5), (298, 2), (299, 4)):
        sizes[e] = rows * part // 12
    o, spans = run_spans(sizes)
    rows = sum(sizes)
    x, q, s = acts_of(rows, k, f"far{rows}")
    active = [e for e in range(E) if sizes[e]]
    y = sbn.bitlinear_grouped(q, s, o, layer.packed, act="silu")
    g = torch.Generator(device="cuda").manual_seed(3)
    dy = torch.randn(rows, n_out, device="cuda", generator=g).to(torch.bfloat16)
    dx, dw = sbn.bitlinear_grouped_grad_x(dy, o, layer.packed), sbn.bitlinear_grouped_grad_w(dy, q, s, o)
    clean(sbn)

    class One:   # the active experts alone
        dense, gamma = [layer.dense[e] for e in active], layer.gamma[active]
    one = One()

    class Dense(list):
        shape = (len(active), n_out, k)
    one.dense = Dense(one.dense)
    ref, tol, _, _ = reference(one, q, s, [spans[e] for e in active], None, "silu", None)
    close(y, ref, tol, "y")
    xd = q.double() * s.double()[:, None] / 127
    for e in active:
        a, b = spans[e]
        d, wd = dy[a:b].double(), layer.dense[e] * layer.gamma[e]
        ref, mag = d @ wd, d.abs() @ wd.abs()
        close(dx[a:b], ref, H * ref.abs() + (1 + H) * (2 * n_out + 4) * U * mag, f"dx {e}")
        close(dw[e], *dw_reference(d, xd[a:b]), f"dw {e}")
        dw[e].zero_()
    assert not any(bool(part.any()) for part in dw.split(50))


@gpu
def test_two_streams_at_once(sbn_lib, cuda_ok):
    """Forward, backward and optimizer steps of two blocks enqueued on two
    streams without any order between them give what they give alone."""
    sbn = _sbn()
    blocks = []
    for i, (rows, k, n_out, n, m) in enumerate(((14, 512, 2056, 6, 8), (700, 640, 1000, 2, 4))):
        layer = Packed(4, n_out, k, n, m, f"two{i}")
        x, q, s = acts_of(rows, k, f"two{i}")
        o, _ = run_spans([rows // 2, 0, rows // 4, rows - rows // 2 - rows // 4])
        g = torch.Generator(device="cuda").manual_seed(i)
        dy = torch.randn(rows, n_out, device="cuda", generator=g).to(torch.bfloat16)
        p = torch.randn(4, n_out, k, device="cuda", generator=g)
        blocks.append((layer, x, q, s, o, dy, p))

    def step(block, opt, stream):
        layer, x, q, s, o, dy, _ = block
        z = torch.empty_like(dy)
        y = sbn.bitlinear_grouped_x(x, o, layer.packed, act="relu2", residual=dy, out_z=z, stream=stream)
        d, db = sbn.act_grad(dy, z, "relu2", offsets=o, stream=stream)
        dx = sbn.bitlinear_grouped_grad_x(d, o, layer.packed, stream=stream)
        dw = sbn.bitlinear_grouped_grad_w(d, q, s, o, stream=stream)
        opt.step([dw], stream=stream)
        return y, z, d, db, dx, dw, sbn.bitlinear_x_act(x, layer.packed.expert(1), act="gelu", residual=dy, stream=stream)

    def opts():
        return [sbn.AdamW([b[-1].clone()], state_bits=8, seed=2) for b in blocks]
    alone = opts()
    want = [[step(b, o, None) for _ in range(5)] for b, o in zip(blocks, alone)]
    clean(sbn)
    both, streams = opts(), [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            got[i].append(step(blocks[i], both[i], streams[i]))
    clean(sbn)
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for x, y in zip(w, g) for a, b in zip(x, y))
    for a, b in zip(alone, both):
        assert torch.equal(a.params[0], b.params[0]) and torch.equal(a.v[0].float(), b.v[0].float())


def test_grouped_dw_workspace_of_two_parts(sbn_lib):
    """The second part of dY s / 127 adds an fp16 array of the padded rows."""
    lib = sbn_lib
    for rows, e, k, n_out in ((64, 4, 256, 64), (64, 4, 256, 65), (1000, 16, 896, 1000), (3, 1024, 128, 9)):
        one, two = (f(rows, e, k, n_out) for f in (lib.sbn_bitlinear_grouped_grad_w_workspace_bytes,
                                                   lib.sbn_bitlinear_grouped_grad_w2_workspace_bytes))
        padded, pitch = (rows + 63 * min(e, rows)) // 64 * 64, -(-n_out // 8) * 8
        assert two - one == padded * pitch * 2
    assert lib.sbn_bitlinear_grouped_grad_w2_workspace_bytes(64, 4, 100, 64) == 0
    assert lib.sbn_bitlinear_grouped_grad_w2_workspace_bytes(0, 4, 128, 64) == 0


@gpu
@pytest.mark.parametrize("n_out", [264, 129])
@pytest.mark.parametrize("spread", [0, 9])
def test_grouped_dw_of_terms_that_cancel(sbn_lib, cuda_ok, n_out, spread):
    """Pairs of rows with opposite gradients and nearly the same activations
    (as two answers to one prompt have them): dW is what is left of them.
    Tolerance, u = 2^-24, n rows: a = dY s / 127 carries two roundings in fp32
    and 2^-22 of itself from its two fp16 parts (half a step of each), or 2^-39 of
    its column's largest; 2 n exact products summed in fp32 in any order, doubled
    for the tensor core's alignment of addends, 4 n u of the sum of |products|;
    one rounding to bf16. One fp16 part, which loses 2^-11 of every term, is 20
    times over it, but stays within dw_reference's tolerance."""
    sbn = _sbn()
    k, sizes = 384, (16, 0, 2, 12, 34)
    o, spans = run_spans(sizes)
    rows = sum(sizes)
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(rows, k, device="cuda", generator=g)
    x[1::2] = x[0::2] * (1 + 2.0 ** -6)
    dy = torch.randn(rows // 2, n_out, device="cuda", generator=g)
    dy = dy * torch.exp2(spread * torch.rand(rows // 2, n_out, device="cuda", generator=g))
    dy = torch.stack([dy, -dy], dim=1).view(rows, n_out).to(torch.bfloat16)
    q, s = sbn.quantize_acts(x.to(torch.bfloat16))
    xd = q.double() * s.double()[:, None] / 127
    one = torch.empty(int(sbn.lib().sbn_bitlinear_grouped_grad_w_workspace_bytes(rows, len(sizes), k, n_out)), dtype=torch.uint8,
                      device="cuda")
    two_parts = sbn.bitlinear_grouped_grad_w(dy, q, s, o)
    one_part = sbn.bitlinear_grouped_grad_w(dy, q, s, o, workspace=one)
    clean(sbn)
    worst = 0.0
    for e, (a, b) in enumerate(spans):
        d, n = dy[a:b].double(), b - a
        ref, tol = dw_reference(d, xd[a:b])
        close(one_part[e], ref, tol, f"one part {e}")
        mag = d.abs().T @ xd[a:b].abs()
        err = ((4 * n + 10) * U + 2.0 ** -22) * mag
        if n:
            err = err + 2.0 ** -39 * d.abs().amax(dim=0)[:, None] * xd[a:b].abs().amax() * n
        tol = H * ref.abs() + (1 + H) * err
        close(two_parts[e], ref, tol, f"two parts {e}")
        if n:
            worst = max(worst, float(((one_part[e].double() - ref).abs() / tol).max()))
    assert worst > 3   # the case tells the two apart


@gpu
def test_adamw_refuses_storage_exchanged_for_one_in_use(sbn_lib, cuda_ok):
    """Two parameters whose storage became one, before the first step or later,
    would be updated by two threads at once."""
    sbn = _sbn()
    a, b = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
    g = [torch.ones(300, device="cuda"), torch.ones(300, device="cuda")]
    for steps in (0, 1):
        opt = sbn.AdamW([a, b])
        for _ in range(steps):
            opt.step(g)
        own, b.data = b.data, a.data
        with pytest.raises(ValueError):
            opt.step(g)
        b.data = torch.ones(900, device="cuda")[10:310]   # one of its own is followed
        opt.step(g)
        clean(sbn)
        assert opt.step_state.tolist() == [steps + 1, 0] and bool((b < 1).all())
        b.data = own


@gpu
def test_adamw_refuses_storage_of_another_type(sbn_lib, cuda_ok):
    """Types of as many bytes: fp32 read as bf16 pairs or whole numbers."""
    sbn = _sbn()
    p, g = torch.ones(300, device="cuda"), [torch.ones(300, device="cuda")]
    opt = sbn.AdamW([p])
    for other in (torch.ones(600, device="cuda", dtype=torch.bfloat16), torch.ones(300, device="cuda", dtype=torch.int32)):
        p.data = other
        with pytest.raises(ValueError):
            opt.step(g)
    p.data = torch.ones(300, device="cuda")
    opt.step(g)
    clean(sbn)
    assert bool((p < 1).all())
