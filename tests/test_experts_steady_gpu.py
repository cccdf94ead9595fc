"""The experts' products where a CTA takes many tiles of several stages each: accumulators, stages and their parities come round
many times.  Whole numbers, whose sums are exact: any element from elsewhere shows."""
import pytest
import torch

import experts_reference as ref

pytestmark = pytest.mark.gpu
HF, F32 = torch.float16, torch.float32


@pytest.fixture(scope="module")
def mfr():
    import moe_finalize_residual_gb300 as m
    yield m
    torch.cuda.synchronize()
    assert m.moe_expert_read_timeouts() == 0


def _whole(g, *shape):
    """Mostly zeros, so that sums of several hundred products stay whole numbers of FP16."""
    v = torch.randint(-2, 3, shape, generator=g, device="cuda", dtype=torch.int8)
    return (v * (torch.rand(shape, generator=g, device="cuda") < 0.5)).to(HF)


def _case(counts, seed, align=1, free=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    off, R = ref.order(counts, align, free)
    return g, off, R, off.cuda(), torch.tensor(counts, dtype=torch.int32).cuda()


def _products(x, w, off, counts):
    """Each expert's rows times its weights, in 64 bits on the GPU."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
    for e, s in ref.spans(off, counts):
        y[s] = x[s].double() @ w[e].double().T
    return y


# Tiles per CTA (152) or pair of CTAs (76), and stages of 64 values a tile:
#   few rows: 1 to 32 rows an expert, 128 values a tile (gated 64)
#   many rows: tiles of up to 256 rows x 256 values (gated 128)
FEW = [17, 0, 3, 32, 1, 9, 20, 31] * 6
MANY = [700, 0, 523, 1, 256, 257, 1030, 90]


@pytest.mark.parametrize("counts,n_in,n_out", [(FEW, 840, 4104), (FEW, 200, 8200), (MANY, 712, 4360), (MANY, 2056, 2568)])
def test_product(mfr, counts, n_in, n_out):
    g, off, R, o, c = _case(counts, n_in, 8, 5)
    x, w = _whole(g, R, n_in), _whole(g, len(counts), n_out, n_in)
    want = _products(x, w, off, counts)
    assert want.abs().max() <= 2048
    assert torch.equal(mfr.moe_expert_matmul(x, w, o, c).double(), want)


@pytest.mark.parametrize("counts,n_in,F", [(FEW, 456, 2056), (MANY, 712, 2184)])
def test_gated_product(mfr, counts, n_in, F):
    g, off, R, o, c = _case(counts, n_in + 1)
    x, w = _whole(g, R, n_in), _whole(g, len(counts), 2 * F, n_in)
    kept = torch.full((R, 2 * F), 7.0, dtype=HF, device="cuda")
    out = mfr.moe_expert_matmul(x, w, o, c, gated=True, gate_up=kept)
    want = _products(x, w, off, counts)
    assert want.abs().max() <= 2048 and torch.equal(kept.double(), want)
    y, err = ref.gate(want[:, :F], want[:, F:])
    finite = y.abs() < 65000  # (a product of two such numbers may pass FP16)
    ref.close("out", out[finite], y[finite], err[finite])
    assert finite.double().mean() > 0.9 and torch.equal(mfr.moe_expert_matmul(x, w, o, c, gated=True), out)


@pytest.mark.parametrize("counts,n_in,n_out", [(FEW, 4104, 840), (MANY, 4360, 712)])
def test_gradient_to_the_rows(mfr, counts, n_in, n_out):
    g, off, R, o, c = _case(counts, n_in + 2, 4, 3)
    d, w = _whole(g, R, n_out), _whole(g, len(counts), n_out, n_in)
    want = _products(d, w.transpose(1, 2), off, counts)
    assert want.abs().max() <= 2048
    assert torch.equal(mfr.moe_expert_matmul_backward(d, None, w, o, c, want_d_weight=False)[0].double(), want)


@pytest.mark.parametrize("counts", [
    [300, 0, 64, 1, 451, 128, 65, 200],               # one CTA a tile
    [900, 0, 64, 1, 1451, 128, 650, 1000, 640, 513],  # pairs
])
@pytest.mark.parametrize("dtype", [HF, F32])
def test_gradient_to_the_weights(mfr, counts, dtype):
    """Reductions of up to 23 stages in a ring of six or four, whole and ragged ones in turn, ten tiles and more a CTA."""
    n_in, n_out = 4104, 3080
    g, off, R, o, c = _case(counts, len(counts), 1, 9)
    x, d = _whole(g, R, n_in), _whole(g, R, n_out)
    x[off[-1]:], d[off[-1]:] = float("nan"), float("nan")
    held = torch.full((len(counts), n_out, n_in), 3.0, device="cuda") if dtype is F32 else None
    _, dw = mfr.moe_expert_matmul_backward(d, x, None, o, c, want_d_rows=False, d_weight=held, d_weight_dtype=dtype, accumulate=dtype is F32)
    assert (R >= 512 * len(counts)) == (len(counts) == 10)
    for e, s in ref.spans(off, counts):
        want = d[s].double().T @ x[s].double()
        assert want.abs().max() <= 2045
        assert torch.equal(dw[e].double(), want + (3 if dtype is F32 else 0)), e


def _fp4(g, *lead):
    """Codes of 0, +-1, +-2 and scales of 1 and 2; their values."""
    table = torch.tensor([0, 2, 4, 10, 12, 0, 0, 0], dtype=torch.uint8, device="cuda")
    pick = lambda: table[torch.randint(0, 8, (*lead[:-1], lead[-1] // 2), generator=g, device="cuda")]  # noqa: E731
    codes = pick() | (pick() << 4)
    sf = torch.tensor([0x38, 0x40], dtype=torch.uint8, device="cuda")[torch.randint(0, 2, (*lead[:-1], lead[-1] // 16), generator=g, device="cuda")]
    return codes, sf, ref.values(codes) * sf.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,n_in,n_out", [(FEW, 832, 2176), (FEW, 1600, 1280), (MANY, 704, 2176), (MANY, 1088, 1280)])
def test_nvfp4_product(mfr, counts, n_in, n_out, gated):
    """Stages of 256 values; the last of a tile holds 64, the scale warps and their tiles come round at different times."""
    g, off, R, o, c = _case(counts, n_in + 3, 1, 4)
    wide = 2 * n_out if gated else n_out
    codes, sf, x = _fp4(g, R, n_in)
    codes[off[-1]:], sf[off[-1]:] = 0x77, 0x7f
    wc, wf, w = _fp4(g, len(counts), wide, n_in)
    tiled = torch.full((len(counts), -(-wide // 128) * 128 * n_in // 16), 0x7f, dtype=torch.uint8, device="cuda")
    tiled[:, ref.tile_at(wide, n_in // 16).cuda()] = wf
    alpha = torch.full((len(counts),), 0.0625, device="cuda")
    out = mfr.moe_expert_matmul_nvfp4(codes, sf, wc, tiled, o, c, alpha=alpha, gated=gated, dtype=HF)
    x[off[-1]:] = 0
    want = _products(x, w, off, counts) / 16
    assert want.abs().max() < 128  # (times 16 at most 2048: exact)
    if not gated:
        assert torch.equal(out.double(), want)
        return
    y, err = ref.gate(want[:, :n_out], want[:, n_out:])
    ref.close("out", out, y, err)


@pytest.mark.parametrize("align", [8, 128])
def test_a_decode_step_in_a_padded_buffer(mfr, align):
    """Few rows an expert, each expert's from a multiple of `align` on: the buffer's rows choose another kernel at 128, and the results
    are the same."""
    counts, n_in, n_out = [1, 0, 2, 7, 1, 0, 0, 3, 16, 1, 5, 0] * 4, 832, 384
    got = {}
    for a in (1, align):
        g, off, R, o, c = _case(counts, 4, a)
        live = ~ref.free_rows(off, counts, R).cuda()
        n = sum(counts)
        some, w = _whole(g, n, n_in), _whole(g, len(counts), 2 * n_out, n_in)
        sc, sf, _ = _fp4(g, n, n_in)
        wc, wf, _ = _fp4(g, len(counts), 2 * n_out, n_in)
        x, codes, scales = torch.full((R, n_in), float("nan"), dtype=HF, device="cuda"), torch.full((R, n_in // 2), 0x77, dtype=torch.uint8, device="cuda"), \
            torch.full((R, n_in // 16), 0x7f, dtype=torch.uint8, device="cuda")
        x[live], codes[live], scales[live] = some, sc, sf
        tiled = torch.zeros(len(counts), 2 * n_out * n_in // 16, dtype=torch.uint8, device="cuda")
        tiled[:, ref.tile_at(2 * n_out, n_in // 16).cuda()] = wf
        y = [mfr.moe_expert_matmul(x, w, o, c), mfr.moe_expert_matmul_nvfp4(codes, scales, wc, tiled, o, c, dtype=HF)]
        y.append(mfr.moe_expert_matmul_backward(y[0].clamp(-2, 2), None, w, o, c, want_d_weight=False)[0])
        assert all((t[~live] == 0).all() for t in y)
        got[a] = [t[live] for t in y]
    assert (mfr.moe_expert_matmul_nvfp4_workspace_bytes(len(counts), R, n_in) > 0) == (align == 128)
    assert all(t.abs().max() <= 2048 and torch.equal(t, u) for t, u in zip(got[1], got[align]))


def test_gradients_on_two_streams_at_once(mfr):
    counts = [300, 5, 0, 250]
    g, off, R, o, c = _case(counts, 8)
    x, w, d = _whole(g, R, 256), _whole(g, 4, 264, 256), _whole(g, R, 264)
    want = _products(d, w.transpose(1, 2), off, counts)
    want_w = torch.stack([d[s].double().T @ x[s].double() for _, s in ref.spans(off, counts)])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [mfr.moe_expert_matmul_backward(d, x, w, o, c, stream=streams[i % 2]) for i in range(12)]
    torch.cuda.synchronize()
    assert want.abs().max() <= 2048 and want_w.abs().max() <= 2048
    assert all(torch.equal(a.double(), want) and torch.equal(b.double(), want_w) for a, b in got)


# ----------------------------------------------------------------------------------------------------------------
# NVFP4 quantisation
# ----------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["row_major", "swizzled_128x4"])
@pytest.mark.parametrize("shape", [(3, 64), (130, 272), (5, 130, 80), (3, 128, 256)])
@pytest.mark.parametrize("masked", [False, True])
def test_quantisation_with_and_without_routes(mfr, layout, shape, masked):
    """Both calls for themselves; back, rows of no route are not read: their codes and scales say something else."""
    g = torch.Generator().manual_seed(sum(shape))
    x, scale = torch.randn(*shape, generator=g).to(HF), 37.25
    lead, H = shape[:-1], shape[-1]
    matrices, rows = (1, *lead) if len(lead) == 1 else lead
    route = torch.arange(matrices * rows, dtype=torch.int32).view(lead)
    if masked:
        route[..., 1::3] = -1
    dead = route < 0
    codes, sf = ref.quantize(x, scale)
    codes[dead], sf[dead] = 0, 0
    x[dead] = float("nan")
    r = route.cuda() if masked else None
    one = torch.tensor([scale]).cuda()
    got, got_sf = mfr.nvfp4_quantize(x.cuda(), one, sf_layout=layout, row_route=r)
    packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
    assert torch.equal(got.cpu(), packed)
    blocks = H // 16
    at = torch.arange(rows * blocks).view(rows, blocks) if layout == "row_major" else ref.tile_at(rows, blocks)
    flat = got_sf.cpu().view(matrices, -1)
    want = torch.zeros(flat.shape, dtype=torch.float64)
    want[:, at] = sf.view(matrices, rows, blocks)
    assert torch.equal(flat.view(torch.float8_e4m3fn).double(), want)
    # back
    flat, spoiled = flat.clone(), got.cpu().clone()
    if masked:
        spoiled[dead] = 0x77
        flat[:, at[dead.view(matrices, rows)[0]]] = 0x7f
    back = mfr.nvfp4_dequantize(spoiled.cuda(), flat.view(got_sf.shape).cuda(), one, sf_layout=layout, row_route=r, dtype=HF).cpu()
    v = (ref.values(packed).unflatten(-1, (-1, 16)) * (sf / scale)[..., None]).flatten(-2)
    assert (back[dead] == 0).all()
    ref.close("values", back, v, 2.0 ** -23 * v.abs())
