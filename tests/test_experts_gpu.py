"""The experts' products on the GPU against their definitions in 64 bits: sizes where tiles end, experts without rows, rows of
no expert that hold NaN, strides, types, and runs of the operators together."""
import pytest
import torch

import experts_reference as ref

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def mfr():
    import moe_finalize_residual_gb300 as m
    yield m
    torch.cuda.synchronize()
    assert m.moe_expert_read_timeouts() == 0


def _dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _case(counts, n, act, seed, align=1, free=0, whole=False):
    """Rows [R, n], NaN where no expert has them, offsets and counts; ``whole``: small whole numbers, whose sums are exact."""
    g = torch.Generator().manual_seed(seed)
    offsets, R = ref.order(counts, align, free)
    x = (torch.randint(-2, 3, (R, n), generator=g).float() if whole else torch.randn(R, n, generator=g)).to(act)
    x[ref.free_rows(offsets, counts, R)] = float("nan")
    return x, offsets, torch.tensor(counts, dtype=torch.int32), g


def _weights(g, E, n, n_in, act, whole=False):
    w = torch.randint(-2, 3, (E, n, n_in), generator=g).float() if whole else torch.randn(E, n, n_in, generator=g) * n_in ** -0.5
    return w.to(act)


COUNTS = [
    ([1], 1, 0),
    ([0, 0, 3], 1, 2),
    ([5, 0, 64, 1], 1, 0),
    ([17, 128, 0, 129, 0], 1, 7),
    ([65, 3, 0, 200], 128, 0),
    ([300], 8, 130),
    ([256, 515, 0, 31], 1, 3),
]


@pytest.mark.parametrize("counts,align,free", COUNTS)
@pytest.mark.parametrize("n_in,n_out", [(64, 256), (8, 8), (200, 264), (72, 520), (1024, 128)])
def test_whole_numbers_are_exact(mfr, counts, align, free, n_in, n_out):
    """Sums of small whole numbers have no rounding: any element taken from elsewhere shows."""
    x, off, cnt, g = _case(counts, n_in, HF, n_in + len(counts), align, free, whole=True)
    w = _weights(g, len(counts), n_out, n_in, HF, whole=True)
    out = mfr.moe_expert_matmul(*_dev(x, w, off, cnt)).cpu()
    want = torch.zeros(x.shape[0], n_out, dtype=torch.float64)
    for e, s in ref.spans(off, counts):
        want[s] = x[s].double() @ w[e].double().T
    assert want.abs().max() <= 4096
    assert torch.equal(out, want.half())


@pytest.mark.parametrize("counts,align,free", COUNTS)
@pytest.mark.parametrize("n_in,n_out", [(64, 256), (8, 8), (200, 264), (520, 72), (1024, 128)])
def test_gradients_of_whole_numbers_are_exact(mfr, counts, align, free, n_in, n_out):
    x, off, cnt, g = _case(counts, n_in, HF, 2 * n_in + len(counts), align, free, whole=True)
    d = torch.randint(-2, 3, (x.shape[0], n_out), generator=g).to(HF)
    d[ref.free_rows(off, counts, x.shape[0])] = float("nan")
    w = _weights(g, len(counts), n_out, n_in, HF, whole=True)
    dx, dw = mfr.moe_expert_matmul_backward(*_dev(d, x, w, off, cnt))
    _, dw32 = mfr.moe_expert_matmul_backward(*_dev(d, x, None, off, cnt), want_d_rows=False, d_weight_dtype=F32)
    want_x, want_w = torch.zeros(x.shape, dtype=torch.float64), torch.zeros(w.shape, dtype=torch.float64)
    for e, s in ref.spans(off, counts):
        want_x[s] = d[s].double() @ w[e].double()
        want_w[e] = d[s].double().T @ x[s].double()
    assert want_x.abs().max() <= 4096 and want_w.abs().max() <= 4096
    assert torch.equal(dx.cpu(), want_x.half())
    assert torch.equal(dw.cpu(), want_w.half())
    assert torch.equal(dw32.cpu(), want_w.float())


@pytest.mark.parametrize("act", [BF, HF])
@pytest.mark.parametrize("counts,align,free", COUNTS[2:])
@pytest.mark.parametrize("gated", [False, True])
def test_forward(mfr, act, counts, align, free, gated):
    n_in, n_out = 328, 168
    x, off, cnt, g = _case(counts, n_in, act, 5, align, free)
    w = _weights(g, len(counts), n_out * (2 if gated else 1), n_in, act)
    kept = torch.full((x.shape[0], 2 * n_out), 7.0, dtype=act).cuda() if gated else None
    out = torch.full((x.shape[0], n_out), 5.0, dtype=act).cuda()
    dx, dw, do, dc = _dev(x, w, off, cnt)
    assert mfr.moe_expert_matmul(dx, dw, do, dc, gated=gated, gate_up=kept, out=out) is out
    zeros = mfr.moe_expert_matmul(dx, dw, do, dc, gated=gated)
    out, zeros, free_row = out.cpu(), zeros.cpu(), ref.free_rows(off, counts, x.shape[0])
    assert (out[free_row] == 5).all() and (zeros[free_row] == 0).all()
    assert torch.equal(out[~free_row], zeros[~free_row])
    for e, s in ref.spans(off, counts):
        y, err = ref.summed(x[s], w[e])
        if gated:
            ref.close("gate_up", kept.cpu()[s], y, err)
            y, err = ref.gate(y[:, :n_out], y[:, n_out:], err[:, :n_out], err[:, n_out:])
        ref.close("out", out[s], y, err)
    if gated:
        assert (kept.cpu()[free_row] == 7).all()


@pytest.mark.parametrize("act", [BF, HF])
@pytest.mark.parametrize("counts,align,free", COUNTS[2:])
def test_backward(mfr, act, counts, align, free):
    n_in, n_out = 168, 328
    x, off, cnt, g = _case(counts, n_in, act, 6, align, free)
    w = _weights(g, len(counts), n_out, n_in, act)
    R = x.shape[0]
    free_row = ref.free_rows(off, counts, R)
    d = torch.randn(R, n_out, generator=g).to(act)
    d[free_row] = float("inf")
    held = torch.randn(w.shape, generator=g)
    dd, dx, dw, do, dc = _dev(d, x, w, off, cnt)
    d_rows, d_weight = mfr.moe_expert_matmul_backward(dd, dx, dw, do, dc)
    kept = torch.full((R, n_in), 5.0, dtype=act).cuda()
    added = held.cuda()
    mfr.moe_expert_matmul_backward(dd, dx, dw, do, dc, d_rows=kept, d_weight=added, accumulate=True)
    d_rows, d_weight, kept, added = d_rows.cpu(), d_weight.cpu(), kept.cpu(), added.cpu()
    assert (d_rows[free_row] == 0).all() and (kept[free_row] == 5).all() and torch.equal(d_rows[~free_row], kept[~free_row])
    for e, s in ref.spans(off, counts):
        y, err = ref.summed(d[s], w[e].T)
        ref.close("d_rows", d_rows[s], y, err)
        y, err = ref.summed(d[s].T, x[s].T)
        ref.close("d_weight", d_weight[e], y, err)
        ref.close("d_weight added", added[e], y + held[e].double(), err)
        if not counts[e]:
            assert (d_weight[e] == 0).all() and torch.equal(added[e], held[e])


# ----------------------------------------------------------------------------------------------------------------
# The gate's gradient
# ----------------------------------------------------------------------------------------------------------------

def _gate_grad(d, g, u):
    """d_g, d_u and the gate's output in 64 bits, with the errors of a few FP32 operations and one exponential each: p and 1 - p
    to (|g| + 8) * 2^-23 relative to the larger of them and 1."""
    d, g, u = d.double(), g.double(), u.double()
    p = torch.where(g >= 0, 1 / (1 + torch.exp(-g)), torch.exp(g) / (1 + torch.exp(g)))
    rel = (g.abs() + 8) * 2.0 ** -23
    dg = d * u * p * (1 + g * (1 - p))
    return (dg, rel * (d * u).abs() * p * (1 + 2 * g.abs())), (d * g * p, rel * (d * g * p).abs()), (g * p * u, rel * (g * p * u).abs())


@pytest.mark.parametrize("act", [BF, HF])
@pytest.mark.parametrize("R,F", [(1, 8), (3, 1000), (130, 72), (33, 4104)])
def test_swiglu_backward(mfr, act, R, F):
    g = torch.Generator().manual_seed(R * F)
    x = (torch.randn(R, 2 * F, generator=g) * 4).to(act)
    x[0, :8] = torch.tensor([0.0, -0.0, 100.0, -100.0, 30.0, -30.0, 1e-3, -1e4]).to(act)
    d = torch.randn(R, F, generator=g).to(act)
    route = torch.arange(R, dtype=torch.int32)
    route[1::3] = -1
    dead = route < 0
    x[dead], d[dead] = float("nan"), float("nan")
    dx, dd, dr = _dev(x, d, route)
    d_x, y = mfr.moe_swiglu_backward(dd, dx, row_route=dr)
    # strided inputs and outputs, in place
    wide = torch.full((R, 2 * F + 16), 3.0, dtype=act).cuda()
    wide[:, 8:8 + 2 * F] = dx
    half = torch.full((R, F + 8), 3.0, dtype=act).cuda()
    half[:, :F] = dd
    mfr.moe_swiglu_backward(half[:, :F], wide[:, 8:8 + 2 * F], row_route=dr, d_gate_up=wide[:, 8:8 + 2 * F], act=half[:, :F])
    assert torch.equal(wide[:, 8:8 + 2 * F], d_x) and torch.equal(half[:, :F], y)
    assert (wide[:, :8] == 3).all() and (wide[:, 8 + 2 * F:] == 3).all() and (half[:, F:] == 3).all()
    only, none = mfr.moe_swiglu_backward(None, dx, want_d_gate_up=False, row_route=dr), mfr.moe_swiglu_backward(dd, dx, want_act=False, row_route=dr)
    assert only[0] is None and none[1] is None and torch.equal(only[1], y) and torch.equal(none[0], d_x)
    d_x, y = d_x.cpu(), y.cpu()
    assert (d_x[dead] == 0).all() and (y[dead] == 0).all()
    live = ~dead
    a, b, c = _gate_grad(d[live], x[live][:, :F], x[live][:, F:])
    ref.close("d_gate", d_x[live][:, :F], *a)
    ref.close("d_up", d_x[live][:, F:], *b)
    ref.close("act", y[live], *c)


# ----------------------------------------------------------------------------------------------------------------
# NVFP4
# ----------------------------------------------------------------------------------------------------------------

def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


@pytest.mark.parametrize("act", [BF, HF])
@pytest.mark.parametrize("layout", ["row_major", "swizzled_128x4"])
@pytest.mark.parametrize("shape", [(1, 16), (3, 64), (130, 272), (129, 9008), (2, 5, 80), (3, 128, 256)])
@pytest.mark.parametrize("scale", [1.0, 37.25])
def test_quantize(mfr, act, layout, shape, scale):
    g = torch.Generator().manual_seed(sum(shape))
    x = (torch.randn(*shape, generator=g) * torch.exp(2 * torch.randn(*shape[:-1], 1, generator=g))).to(act)
    x[..., 0, :16] = 0.0
    x.reshape(-1, shape[-1])[-1, :4] = torch.tensor([1e4, -1e4, 1e-4, -0.0]).to(act)
    lead, H = shape[:-1], shape[-1]
    matrices, rows = (1, shape[0]) if len(shape) == 2 else shape[:2]
    route = torch.arange(matrices * rows, dtype=torch.int32).view(lead)
    if len(shape) == 2 and rows > 2:
        route[1] = -1
    codes, sf = ref.quantize(x, scale)
    codes[route < 0], sf[route < 0] = 0, 0
    x[route < 0] = float("nan")
    dx, ds, dr = _dev(x, torch.tensor([scale]), route)
    for r in (None, dr) if not (route < 0).any() else (dr,):
        got, got_sf = mfr.nvfp4_quantize(dx, ds, sf_layout=layout, row_route=r)
        back = mfr.nvfp4_dequantize(got, got_sf, ds, sf_layout=layout, row_route=r, dtype=act)
    assert got_sf.numel() == mfr.nvfp4_sf_bytes(rows, H, layout, matrices)
    flat = got_sf.cpu().view(torch.float8_e4m3fn).double().view(matrices, -1)
    want = sf.reshape(matrices, rows, H // 16)
    if layout == "row_major":
        assert torch.equal(flat, want.flatten(1))
    else:
        tiled = torch.zeros(matrices, flat.shape[1], dtype=torch.float64)  # zeros behind the last row and block
        tiled[:, ref.tile_at(rows, H // 16)] = want
        assert torch.equal(flat, tiled)
    assert torch.equal(got.cpu(), _pack(codes))
    v = ref.values(_pack(codes)).unflatten(-1, (-1, 16)) * (sf / scale)[..., None]
    ref.close("values", back.cpu(), v.flatten(-2), 2.0 ** -23 * v.flatten(-2).abs())


def test_quantize_of_what_is_not_finite(mfr):
    x = torch.ones(2, 48, dtype=BF)
    x[0, 3], x[0, 20], x[1, 40] = float("nan"), float("inf"), float("-inf")
    ds = torch.tensor([2.0]).cuda()
    codes, sf = mfr.nvfp4_quantize(x.cuda(), ds)
    sf = sf.cpu().view(torch.float8_e4m3fn).float()
    assert torch.isnan(sf[0, 0]) and (sf[0, 1], sf[1, 2]) == (448, 448) and torch.isfinite(sf.flatten()[1:]).all()
    v = mfr.nvfp4_dequantize(codes, codes.new_tensor(sf.to(torch.float8_e4m3fn).view(torch.uint8).tolist()), ds).cpu().float()
    assert torch.isnan(v[0, :16]).all() and v[0, 20] == 6 * 448 / 2 and v[1, 40] == -6 * 448 / 2 and (v[0, 32:] != 0).all()


def _nvfp4_case(counts, n_in, n, seed, align=1, free=0, whole=False):
    """Random codes and scales; ``whole``: scales 1 and 2, whose sums are exact."""
    g = torch.Generator().manual_seed(seed)
    offsets, R = ref.order(counts, align, free)
    E = len(counts)
    def some(*lead):
        c = torch.randint(0, 256, (*lead, n_in // 2), generator=g, dtype=torch.uint8)
        if whole:  # values 0, +-1, +-2 only
            table = torch.tensor([0, 2, 4, 10, 12], dtype=torch.uint8)
            c = table[torch.randint(0, 5, (*lead, n_in // 2), generator=g)] | (table[torch.randint(0, 5, (*lead, n_in // 2), generator=g)] << 4)
        f = torch.tensor([1.0, 2.0])[torch.randint(0, 2, (*lead, n_in // 16), generator=g)] if whole else \
            torch.exp(torch.randn(*lead, n_in // 16, generator=g))
        return c, f.to(torch.float8_e4m3fn)
    c, f = some(R)
    free_row = ref.free_rows(offsets, counts, R)
    c[free_row] = 0x77
    f.view(torch.uint8)[free_row] = 0x7f  # not a number
    wc, wf = some(E, n)
    bytes_ = -(-n // 128) * 128 * -(-n_in // 64) * 4
    tiled = torch.full((E, bytes_), 0x7f, dtype=torch.uint8)  # behind the last row: anything
    tiled[:, ref.tile_at(n, n_in // 16)] = wf.view(torch.uint8)
    x = ref.values(c).unflatten(-1, (-1, 16)) * f.double()[..., None]
    w = ref.values(wc).unflatten(-1, (-1, 16)) * wf.double()[..., None]
    return c, f.view(torch.uint8), wc, tiled, offsets, torch.tensor(counts, dtype=torch.int32), x.flatten(-2), w.flatten(-2), g


@pytest.mark.parametrize("counts,align,free", COUNTS)
@pytest.mark.parametrize("n_in,n_out", [(64, 256), (256, 8), (320, 264), (576, 520), (1024, 128)])
def test_nvfp4_whole_numbers_are_exact(mfr, counts, align, free, n_in, n_out):
    c, f, wc, wf, off, cnt, x, w, _ = _nvfp4_case(counts, n_in, n_out, n_in + len(counts), align, free, whole=True)
    out = mfr.moe_expert_matmul_nvfp4(*_dev(c, f, wc, wf, off, cnt), dtype=HF).cpu()
    want = torch.zeros(x.shape[0], n_out, dtype=torch.float64)
    for e, s in ref.spans(off, counts):
        want[s] = x[s] @ w[e].T
    assert want.abs().max() <= 2048
    assert torch.equal(out, want.half())


@pytest.mark.parametrize("act", [BF, HF])
@pytest.mark.parametrize("counts,align,free", COUNTS[2:])
@pytest.mark.parametrize("gated", [False, True])
def test_nvfp4_product(mfr, act, counts, align, free, gated):
    n_in, n_out = 832, 256
    c, f, wc, wf, off, cnt, x, w, g = _nvfp4_case(counts, n_in, 2 * n_out if gated else n_out, 9, align, free)
    alpha = torch.rand(len(counts), generator=g) * 0.01
    args = _dev(c, f, wc, wf, off, cnt)
    out = torch.full((x.shape[0], n_out), 5.0, dtype=act).cuda()
    mfr.moe_expert_matmul_nvfp4(*args, alpha=alpha.cuda(), gated=gated, out=out)
    zeros = mfr.moe_expert_matmul_nvfp4(*args, alpha=alpha.cuda(), gated=gated, dtype=act).cpu()
    out, free_row = out.cpu(), ref.free_rows(off, counts, x.shape[0])
    assert (out[free_row] == 5).all() and (zeros[free_row] == 0).all() and torch.equal(out[~free_row], zeros[~free_row])
    for e, s in ref.spans(off, counts):
        y, err = ref.summed(x[s], w[e])
        a = alpha[e].double()
        y, err = y * a, err * a + 2.0 ** -24 * (y * a).abs()
        if gated:
            y, err = ref.gate(y[:, :n_out], y[:, n_out:], err[:, :n_out], err[:, n_out:])
        ref.close("out", out[s], y, err)
