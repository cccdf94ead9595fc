"""The experts' products as they are used: strided views, calls without counts, far offsets, other streams, captured graphs, two
calls at once, what is refused, and runs of the operators together, forward and back, against 64 bits."""
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


def _whole(g, *shape, dtype=HF):
    return torch.randint(-2, 3, shape, generator=g).to(dtype)


def _case(counts, n_in, n_out, seed, align=1, free=0):
    g = torch.Generator().manual_seed(seed)
    off, R = ref.order(counts, align, free)
    x, w, d = _whole(g, R, n_in), _whole(g, len(counts), n_out, n_in), _whole(g, R, n_out)
    return x, w, d, off, torch.tensor(counts, dtype=torch.int32)


def _want(x, w, off, counts):
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64)
    for e, s in ref.spans(off, counts):
        y[s] = x[s].double() @ w[e].double().T
    return y


def test_strided_rows_weights_and_outputs(mfr):
    counts = [3, 0, 140, 17]
    x, w, d, off, cnt = _case(counts, 72, 136, 1)
    R = x.shape[0]
    wide_x, wide_w = torch.full((R, 96), 9.0, dtype=HF).cuda(), torch.full((4, 150, 80), 9.0, dtype=HF).cuda()
    wide_d, wide_o, wide_dx = (torch.full((R, n), 9.0, dtype=HF).cuda() for n in (152, 152, 96))
    wide_x[:, 8:80], wide_w[:, 8:144, :72], wide_d[:, 16:] = x.cuda(), w.cuda(), d.cuda()
    vx, vw, vd, vo, vdx = wide_x[:, 8:80], wide_w[:, 8:144, :72], wide_d[:, 16:], wide_o[:, 8:144], wide_dx[:, 16:88]
    mfr.moe_expert_matmul(vx, vw, off.cuda(), cnt.cuda(), out=vo)
    _, dw = mfr.moe_expert_matmul_backward(vd, vx, vw, off.cuda(), cnt.cuda(), d_rows=vdx)
    want = _want(x, w, off, counts)
    assert torch.equal(vo.cpu(), want.half())
    assert (wide_o[:, :8] == 9).all() and (wide_o[:, 144:] == 9).all() and (wide_dx[:, :16] == 9).all() and (wide_dx[:, 88:] == 9).all()
    for e, s in ref.spans(off, counts):
        assert torch.equal(vdx.cpu()[s], (d[s].double() @ w[e].double()).half())
        assert torch.equal(dw.cpu()[e], (d[s].double().T @ x[s].double()).half())


@pytest.mark.parametrize("n_in,n_out", [(264, 512), (512, 24), (136, 264)])
@pytest.mark.parametrize("counts", [[700, 0, 523, 1, 256, 257], [1100, 1, 523], [1024, 640], [0, 2051]])
def test_many_rows_an_expert(mfr, counts, n_in, n_out):
    """Several tiles of rows, by pairs of CTAs (the weights' gradient in all but the first), with experts of one row and of none."""
    x, w, d, off, cnt = _case(counts, n_in, n_out, 2)
    args = [t.cuda() for t in (d, x, w, off, cnt)]
    out = mfr.moe_expert_matmul(*args[1:]).cpu()
    dx, dw = (t.cpu() for t in mfr.moe_expert_matmul_backward(*args))
    _, dw32 = mfr.moe_expert_matmul_backward(*args[:2], None, *args[3:], want_d_rows=False, d_weight=torch.full(w.shape, 3.0).cuda(), accumulate=True)
    want = _want(x, w, off, counts)
    assert want.abs().max() <= 2048 and torch.equal(out, want.half())
    assert torch.equal(dw32.cpu() - 3, dw.float()) and dw.abs().max() <= 2048 and (dw[torch.tensor(counts) == 0] == 0).all()
    for e, s in ref.spans(off, counts):
        assert torch.equal(dx[s], (d[s].double() @ w[e].double()).half())
        assert torch.equal(dw[e], (d[s].double().T @ x[s].double()).half())


@pytest.mark.parametrize("most", [3, 70])
def test_as_many_experts_as_there_may_be(mfr, most):
    g = torch.Generator().manual_seed(most)
    counts = torch.randint(0, most, (1024,), generator=g)
    counts[::7] = 0
    counts = counts.tolist()
    x, w, d, off, cnt = _case(counts, 64, 64, most)
    args = [t.cuda() for t in (d, x, w, off, cnt)]
    out = mfr.moe_expert_matmul(*args[1:]).cpu()
    dx, dw = (t.cpu() for t in mfr.moe_expert_matmul_backward(*args))
    assert torch.equal(out, _want(x, w, off, counts).half())
    assert torch.equal(dx, _want(d, w.transpose(1, 2), off, counts).half())
    of = torch.repeat_interleave(torch.arange(1024), torch.tensor(counts))
    want = torch.zeros(1024, 64 * 64, dtype=torch.float64).index_add_(0, of, (d.double()[:, :, None] * x.double()[:, None, :]).flatten(1))
    assert torch.equal(dw, want.view(1024, 64, 64).half())
    # the same values in NVFP4: codes of whole numbers, every scale one
    code = torch.tensor([12, 10, 0, 2, 4], dtype=torch.uint8)  # of -2 .. 2
    pack = lambda t: (lambda c: c[..., 0::2] | (c[..., 1::2] << 4))(code[(t.double() + 2).long()])  # noqa: E731
    ones = torch.full((1024, 128 * 4), 0x38, dtype=torch.uint8)
    q = mfr.moe_expert_matmul_nvfp4(pack(x).cuda(), torch.full((x.shape[0], 4), 0x38, dtype=torch.uint8).cuda(), pack(w).cuda(), ones.cuda(),
                                    *args[3:], dtype=HF).cpu()
    assert torch.equal(q, out)


def test_without_counts_every_row_up_to_the_next_expert(mfr):
    x, w, d, off, _ = _case([8, 0, 40], 64, 64, 3)
    args = [t.cuda() for t in (x, w, off)]
    assert torch.equal(mfr.moe_expert_matmul(*args).cpu(), _want(x, w, off, [8, 0, 40]).half())
    dw = mfr.moe_expert_matmul_backward(d.cuda(), *args, want_d_rows=False)[1].cpu()
    assert torch.equal(dw[2], (d[8:].double().T @ x[8:].double()).half()) and (dw[1] == 0).all()


def test_no_rows_at_all(mfr):
    x, w, d = torch.empty(0, 64, dtype=BF).cuda(), torch.ones(3, 128, 64, dtype=BF).cuda(), torch.empty(0, 128, dtype=BF).cuda()
    off = torch.zeros(4, dtype=torch.int32).cuda()
    assert mfr.moe_expert_matmul(x, w, off).shape == (0, 128)
    dx, dw = mfr.moe_expert_matmul_backward(d, x, w, off)
    assert dx.shape == (0, 64) and (dw == 0).all() and dw.shape == w.shape
    # rows, but none of any expert
    x, d = torch.full((5, 64), float("nan"), dtype=BF).cuda(), torch.full((5, 128), float("nan"), dtype=BF).cuda()
    assert (mfr.moe_expert_matmul(x, w, off) == 0).all()
    dx, dw = mfr.moe_expert_matmul_backward(d, x, w, off)
    assert (dx == 0).all() and (dw == 0).all()


def test_wrong_offsets_touch_no_row_outside(mfr):
    """Device data that contradicts the call is cut to its rows; what is written behind them shows in the guard."""
    x, w, d, _, _ = _case([40], 64, 64, 4)
    for off, cnt in (([-5, 30, 1000], [1000, 1000]), ([2000000000, 2147483647, 5], [2147483647, -3]), ([10, 5, 0], [-1, 2])):
        guard = torch.full((120, 64), 7.0, dtype=HF).cuda()
        mfr.moe_expert_matmul(x.cuda(), w.cuda().expand(2, 64, 64).contiguous(), torch.tensor(off, dtype=torch.int32).cuda(),
                              torch.tensor(cnt, dtype=torch.int32).cuda(), out=guard[40:80])
        mfr.moe_expert_matmul_backward(d.cuda(), x.cuda(), w.cuda().expand(2, 64, 64).contiguous(), torch.tensor(off, dtype=torch.int32).cuda(),
                                       torch.tensor(cnt, dtype=torch.int32).cuda(), d_rows=guard[40:80])
        assert (guard[:40] == 7).all() and (guard[80:] == 7).all()
        codes, sf = torch.zeros(60, 32, dtype=torch.uint8).cuda(), torch.zeros(60, 4, dtype=torch.uint8).cuda()
        wc, ws = torch.zeros(2, 64, 32, dtype=torch.uint8).cuda(), torch.zeros(2, 512, dtype=torch.uint8).cuda()
        space = torch.full((mfr.moe_expert_matmul_nvfp4_workspace_bytes(2, 60, 64) + 4096,), 9, dtype=torch.uint8).cuda()
        assert space.numel() > 4096
        mfr.moe_expert_matmul_nvfp4(codes, sf, wc, ws, torch.tensor(off, dtype=torch.int32).cuda(), torch.tensor(cnt, dtype=torch.int32).cuda(),
                                    out=guard[40:100], workspace=space)
        assert (guard[:40] == 7).all() and (guard[100:] == 7).all() and (space[-4096:] == 9).all()


def test_elements_behind_two_to_the_31(mfr):
    """Rows whose elements lie behind 2^31, of every tensor of rows."""
    R, n = 270000, 8192
    counts, off = [3, 300], torch.tensor([0, R - 310, R], dtype=torch.int32)
    g = torch.Generator().manual_seed(5)
    x, d = torch.zeros(R, n, dtype=HF, device="cuda"), torch.empty(R, n, dtype=HF, device="cuda")
    hx, hw, hd = _whole(g, 303, n), _whole(g, 2, 64, n) * (torch.rand(2, 64, n, generator=g) < 0.02), _whole(g, 303, 64)
    at = torch.cat([torch.arange(3), torch.arange(R - 310, R - 10)])
    x[at.cuda()] = hx.cuda()
    cnt = torch.tensor(counts, dtype=torch.int32)
    out = mfr.moe_expert_matmul(x, hw.cuda(), off.cuda(), cnt.cuda()).cpu()
    dd = torch.zeros(R, 64, dtype=HF, device="cuda")
    dd[at.cuda()] = hd.cuda()
    mfr.moe_expert_matmul_backward(dd, x, hw.cuda(), off.cuda(), cnt.cuda(), d_rows=d, want_d_weight=False)
    dx = d[at.cuda()].cpu()
    for e, s in ((0, slice(0, 3)), (1, slice(3, 303))):
        assert torch.equal(out[at[s]], (hx[s].double() @ hw[e].double().T).half())
        assert torch.equal(dx[s], (hd[s].double() @ hw[e].double()).half())
    scale = torch.ones(1).cuda()
    codes, sf = mfr.nvfp4_quantize(x, scale)
    back = mfr.nvfp4_dequantize(codes, sf, scale, dtype=HF)
    want, want_sf = ref.quantize(hx, 1.0)
    assert torch.equal(codes[at.cuda()].cpu(), want[..., 0::2] | (want[..., 1::2] << 4))
    assert torch.equal(back[at.cuda()].cpu().double(), ref.values(codes[at.cuda()].cpu()) * want_sf.repeat_interleave(16, 1))


def _nvfp4_weights(mfr, w, g):
    return mfr.nvfp4_quantize(w, g, sf_layout="swizzled_128x4")


def test_nvfp4_rows_and_weights_as_the_framework_makes_them(mfr):
    """The finalize's NVFP4 output, dispatched with its scales, times weights quantised here."""
    T, K, E, H, F = 37, 4, 16, 512, 256
    g = torch.Generator().manual_seed(6)
    logits = torch.randn(T, E, generator=g).cuda()
    part = mfr.Partial(torch.randn(T, H, generator=g).to(BF).cuda(), torch.arange(T, dtype=torch.int32)[:, None].cuda())
    gx, gw = torch.tensor([448.0]).cuda(), torch.tensor([448.0 * 6 / 4]).cuda()
    _, normed, codes, sf = mfr.moe_finalize_fused([part], torch.randn(T, H, generator=g).to(BF).cuda(), torch.ones(H, dtype=BF).cuda(),
                                                  quant_mode="nvfp4", quant_scale=gx)
    codes, sf = codes.view(T, H // 2), sf.view(T, H // 16)
    own_codes, own_sf = mfr.nvfp4_quantize(normed, gx)
    assert torch.equal(codes, own_codes) and torch.equal(sf, own_sf)  # the same recipe, bit for bit
    r = mfr.moe_route(logits, K, row_align=8)
    x, xs = mfr.moe_dispatch(codes, r.perm_idx, row_route=r.row_route), mfr.moe_dispatch(sf, r.perm_idx, row_route=r.row_route)
    w = (torch.randn(E, 2 * F, H, generator=g) * H ** -0.5).to(BF)
    wc, ws = _nvfp4_weights(mfr, w.cuda(), gw)
    assert wc.shape == (E, 2 * F, H // 2) and ws.shape == (E, 2 * F * H // 16)
    alpha = (1 / (gx * gw)).expand(E).contiguous()
    out = mfr.moe_expert_matmul_nvfp4(x, xs, wc, ws, r.expert_offsets, r.expert_counts, alpha=alpha, gated=True).cpu()
    xv = ref.values(x.cpu()) * xs.cpu().view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    wcodes, wsf = ref.quantize(w, float(gw))
    wv = ref.values(wcodes[..., 0::2] | (wcodes[..., 1::2] << 4)) * wsf.repeat_interleave(16, 2)
    counts = r.expert_counts.cpu().tolist()
    for e, s in ref.spans(r.expert_offsets.cpu(), counts):
        y, err = ref.summed(xv[s], wv[e])
        a = alpha[e].double().cpu()
        y, err = y * a, err * a + 2.0 ** -24 * (y * a).abs()
        y, err = ref.gate(y[:, :F], y[:, F:], err[:, :F], err[:, F:])
        ref.close("out", out[s], y, err)


@pytest.mark.parametrize("counts", [[3, 0, 20, 1], [400, 0, 129, 193, 1]])
@pytest.mark.parametrize("n_in", [512, 576])
def test_nvfp4_scales_from_any_boundary(mfr, counts, n_in):
    """Scales on 4 bytes, not 16; many and few rows."""
    g = torch.Generator().manual_seed(7)
    off, R = ref.order(counts)
    E, n = len(counts), 256
    codes, wc = (torch.randint(0, 256, s, generator=g, dtype=torch.uint8) for s in ((R, n_in // 2), (E, n, n_in // 2)))
    sf = torch.randint(40, 60, (R * (n_in // 16) + 4,), generator=g, dtype=torch.uint8)
    ws = torch.randint(40, 60, (E, n * (n_in // 16)), generator=g, dtype=torch.uint8)
    shifted = sf.cuda()[4:].view(R, n_in // 16)
    assert shifted.data_ptr() % 16 == 4
    args = [t.cuda() for t in (wc, ws, off, torch.tensor(counts, dtype=torch.int32))]
    for gated in (False, True):
        a = mfr.moe_expert_matmul_nvfp4(codes.cuda(), shifted, *args, gated=gated)
        b = mfr.moe_expert_matmul_nvfp4(codes.cuda(), shifted.clone(), *args, gated=gated)
        assert torch.equal(a, b)
    f8 = lambda t: t.view(torch.float8_e4m3fn).double()  # noqa: E731
    x = ref.values(codes) * f8(sf[4:].view(R, -1)).repeat_interleave(16, 1)
    w = ref.values(wc) * f8(ws[:, ref.tile_at(n, n_in // 16)]).repeat_interleave(16, 2)
    out = mfr.moe_expert_matmul_nvfp4(codes.cuda(), shifted, *args).cpu()
    for e, s in ref.spans(off, counts):
        ref.close("out", out[s], *ref.summed(x[s], w[e]))


def test_other_streams_and_two_calls_at_once(mfr):
    counts = [300, 5, 0, 250]
    x, w, d, off, cnt = _case(counts, 256, 256, 8)
    args = [t.cuda() for t in (x, w, off, cnt)]
    want = _want(x, w, off, counts).half()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(12):
        outs.append(mfr.moe_expert_matmul(*args, stream=streams[i % 2]))
        outs.append(mfr.moe_expert_matmul_backward(d.cuda(), *args, stream=streams[(i + 1) % 2])[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), want) for o in outs[0::2]) and all(torch.equal(o, outs[1]) for o in outs[1::2])


def test_captured_and_replayed(mfr):
    """A layer's products and gradients in a graph, replayed on new inputs and new row counts, beside eager calls."""
    E, n_in, F = 4, 128, 64
    g = torch.Generator().manual_seed(9)
    R = 200
    x, w, d = torch.zeros(R, n_in, dtype=HF).cuda(), _whole(g, E, 2 * F, n_in).cuda(), _whole(g, R, F).cuda()
    off, cnt, route = torch.zeros(E + 1, dtype=torch.int32).cuda(), torch.zeros(E, dtype=torch.int32).cuda(), torch.zeros(R, dtype=torch.int32).cuda()
    scale = torch.ones(1).cuda()

    def step():
        kept = torch.zeros(R, 2 * F, dtype=HF, device="cuda")
        y = mfr.moe_expert_matmul(x, w, off, cnt, gated=True, gate_up=kept)
        dg, act = mfr.moe_swiglu_backward(d, kept, row_route=route)
        dx, dw = mfr.moe_expert_matmul_backward(dg, x, w, off, cnt)
        codes, sf = mfr.nvfp4_quantize(x, scale)
        wc, ws = mfr.nvfp4_quantize(w, scale, sf_layout="swizzled_128x4")
        q = mfr.moe_expert_matmul_nvfp4(codes, sf, wc, ws, off, cnt, dtype=HF)
        return y, dg, act, dx, dw, q, mfr.nvfp4_dequantize(codes, sf, scale, dtype=HF)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed, counts in ((1, [50, 0, 100, 50]), (2, [0, 0, 0, 200]), (3, [1, 1, 1, 1])):
        gen = torch.Generator().manual_seed(seed)
        new_off, _ = ref.order(counts)
        x.copy_(_whole(gen, R, n_in))
        off.copy_(new_off)
        cnt.copy_(torch.tensor(counts, dtype=torch.int32))
        route.copy_(torch.where(torch.arange(R) < sum(counts), torch.arange(R), -1).int())
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager))
        y = _want(x.cpu(), w.cpu(), new_off, counts)
        got = held[0].cpu()
        live = slice(0, sum(counts))
        ref.close("out", got[live], *ref.gate(y[live, :F], y[live, F:]))


def test_the_same_from_run_to_run(mfr):
    g = torch.Generator().manual_seed(10)
    counts = [1000, 0, 333, 7]
    off, R = ref.order(counts)
    x, w, d = (torch.randn(*s, generator=g).to(BF).cuda() for s in ((R, 512), (4, 384, 512), (R, 384)))
    args = (x, w, off.cuda(), torch.tensor(counts, dtype=torch.int32).cuda())
    first = (mfr.moe_expert_matmul(*args), *mfr.moe_expert_matmul_backward(d, *args, d_weight_dtype=F32))
    for _ in range(5):
        again = (mfr.moe_expert_matmul(*args), *mfr.moe_expert_matmul_backward(d, *args, d_weight_dtype=F32))
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_values_that_are_not_finite_stay_in_their_rows(mfr):
    counts = [20, 150]
    x, w, d, off, cnt = _case(counts, 128, 128, 11)
    clean = mfr.moe_expert_matmul(*[t.cuda() for t in (x, w, off, cnt)]).cpu()
    x[5, 3], x[60, 9], w[1, 7, 2] = float("nan"), float("inf"), float("nan")
    out = mfr.moe_expert_matmul(*[t.cuda() for t in (x, w, off, cnt)]).cpu()
    assert torch.isnan(out[5]).all() and not torch.isfinite(out[60][w[1, :, 9] != 0]).any() and torch.isnan(out[20:, 7]).all()
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[5], keep[60], keep[20:, 7] = False, False, False
    assert torch.equal(out[keep], clean[keep])


def test_gradients_are_the_differences(mfr):
    """The product is linear: its change over any step, weighed by d_out, is the gradient times the step, exactly for whole numbers.
    The gate's change over a small one, in 64 bits, is its gradient to the second order."""
    counts = [30, 0, 170]
    x, w, d, off, cnt = _case(counts, 64, 40, 12)
    g = torch.Generator().manual_seed(13)
    sx, sw = _whole(g, *x.shape), _whole(g, *w.shape)
    args = [t.cuda() for t in (d, x, w, off, cnt)]
    dx, _ = mfr.moe_expert_matmul_backward(*args)
    _, dw = mfr.moe_expert_matmul_backward(*args, want_d_rows=False, d_weight_dtype=F32)
    f = lambda x, w: mfr.moe_expert_matmul(x.cuda(), w.cuda(), args[3], args[4]).cpu().double()  # noqa: E731
    assert (d.double() * (f(x + sx, w) - f(x, w))).sum() == (dx.cpu().double() * sx.double()).sum()
    assert (d.double() * (f(x, w + sw) - f(x, w))).sum() == (dw.cpu().double() * sw.double()).sum()
    # the gate
    gu, do = torch.randn(50, 32, generator=g).to(HF), torch.randn(50, 16, generator=g).to(HF)
    grad = mfr.moe_swiglu_backward(do.cuda(), gu.cuda())[0].cpu().double()
    h = 1e-4
    for i in range(32):
        step = torch.zeros(32, dtype=torch.float64)
        step[i] = h
        y = [ref.silu((gu.double() + s * step)[:, :16]) * (gu.double() + s * step)[:, 16:] for s in (1, -1)]
        want = (do.double() * (y[0] - y[1])).sum(1) / (2 * h)
        # half a step of FP16, the third derivative (silu's is below 0.6) over h^2 / 6, the operations in FP32
        off_by = 2.0 ** -11 * want.abs() + 2.0 ** -24 + (do.double().abs().sum(1) * gu.double().abs().amax(1)) * (0.1 * h * h + 2.0 ** -18)
        assert ((grad[:, i] - want).abs() <= off_by).all()


@pytest.mark.parametrize("act,T,masked", [(BF, 50, False), (HF, 333, True), (BF, 1, False)])
def test_a_layer_forward_and_back(mfr, act, T, masked):
    """route -> dispatch -> gated product -> product -> finalize, and every gradient back to the tokens and the weights."""
    E, K, H, F = 8, 3, 256, 128
    g = torch.Generator().manual_seed(T)
    logits = torch.randn(T, E, generator=g)
    if masked:
        logits[torch.rand(T, E, generator=g) < 0.5] = float("-inf")
    x, d = torch.randn(T, H, generator=g).to(act), torch.randn(T, H, generator=g).to(act)
    w1, w2 = (torch.randn(E, 2 * F, H, generator=g) * H ** -0.5).to(act), (torch.randn(E, H, F, generator=g) * F ** -0.5).to(act)
    dev = [t.cuda() for t in (logits, x, d, w1, w2)]
    r = mfr.moe_route(dev[0], K, row_align=4)
    at = (r.expert_offsets, r.expert_counts)
    rows = mfr.moe_dispatch(dev[1], r.perm_idx, row_route=r.row_route)
    kept = torch.empty(rows.shape[0], 2 * F, dtype=act, device="cuda")
    mid = torch.empty(rows.shape[0], F, dtype=act, device="cuda")
    mfr.moe_expert_matmul(rows, dev[3], *at, gated=True, gate_up=kept, out=mid)
    part = mfr.Partial(mfr.moe_expert_matmul(mid, dev[4], *at), r.perm_idx, r.expert_scale)
    y = mfr.moe_finalize_routed([part])
    d_rows, d_scale = mfr.moe_finalize_routed_backward(dev[2], part, row_route=r.row_route)
    d_mid, _ = mfr.moe_expert_matmul_backward(d_rows, None, dev[4], *at, want_d_weight=False)
    d_kept, again = mfr.moe_swiglu_backward(d_mid, kept, row_route=r.row_route)
    _, d_w2 = mfr.moe_expert_matmul_backward(d_rows, again, None, *at, want_d_rows=False, d_weight_dtype=F32)
    d_in, d_w1 = mfr.moe_expert_matmul_backward(d_kept, rows, dev[3], *at, d_weight_dtype=F32)
    d_x = mfr.moe_finalize_routed([mfr.Partial(d_in, r.perm_idx)])
    # the same in 64 bits, the weights of the routes as they were rounded
    ids, scale = r.expert_ids.cpu().long(), r.expert_scale.cpu().double()
    X, W1, W2, S = (t.double().requires_grad_() for t in (x, w1, w2, scale))
    out = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        h = X[t] @ W1[e].T
        out = out.index_add(0, t, (ref.silu(h[:, :F]) * h[:, F:]) @ W2[e].T * S[t, k][:, None])
    (out * d.double()).sum().backward()
    # Each value is rounded to the type at most six times on its way (one rounding a step); each is off by u at most, carried on
    # by steps that keep norms within a factor of two here (random weights of unit gain, a gate of slope at most 1.1).
    share = 6 * 2 * ref.U[act]
    for name, got, want in (("y", y, out.detach()), ("d_x", d_x, X.grad), ("d_w1", d_w1, W1.grad), ("d_w2", d_w2, W2.grad),
                            ("d_scale", d_scale, S.grad * (ids >= 0))):
        assert torch.isfinite(got).all(), name
        assert (got.cpu().double() - want).norm() <= share * want.norm(), name


def test_refusals_on_the_gpu(mfr):
    x, w, o = torch.zeros(4, 64, dtype=BF).cuda(), torch.zeros(2, 128, 64, dtype=BF).cuda(), torch.zeros(3, dtype=torch.int32).cuda()
    d, s, c = torch.zeros(4, 128, dtype=BF).cuda(), torch.ones(1).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    u8 = lambda *n: torch.zeros(*n, dtype=torch.uint8).cuda()  # noqa: E731
    wrong = [lambda: mfr.moe_expert_matmul(x, w.half(), o), lambda: mfr.moe_expert_matmul(x, w[:, :, :32], o),
             lambda: mfr.moe_expert_matmul(x.t(), w, o), lambda: mfr.moe_expert_matmul(x, w, o.long()), lambda: mfr.moe_expert_matmul(x, w, o[:2]),
             lambda: mfr.moe_expert_matmul(x, w, o, c[:1]), lambda: mfr.moe_expert_matmul(x, w, o.cpu()),
             lambda: mfr.moe_expert_matmul(x, w, o, out=d.half()), lambda: mfr.moe_expert_matmul(x, w, o, gated=True, gate_up=d[:3]),
             lambda: mfr.moe_expert_matmul(x.float(), w.float(), o), lambda: mfr.moe_expert_matmul_backward(d[:, :64], x, w, o),
             lambda: mfr.moe_expert_matmul_backward(d, x[:3], w, o), lambda: mfr.moe_expert_matmul_backward(d, x, w, o, d_weight=w.half()),
             lambda: mfr.moe_expert_matmul_backward(d, x, w, o, d_weight=w[:, :, :32]), lambda: mfr.moe_expert_matmul_backward(d, x, w, o, d_rows=d),
             lambda: mfr.moe_expert_matmul_backward(d, x, w, o, d_weight_dtype=torch.float64), lambda: mfr.moe_expert_matmul_backward(d, x, w, None),
             lambda: mfr.moe_swiglu_backward(x, d.half()), lambda: mfr.moe_swiglu_backward(x, d, row_route=o),
             lambda: mfr.nvfp4_quantize(x.float(), s), lambda: mfr.nvfp4_quantize(x, s.cpu()), lambda: mfr.nvfp4_quantize(x, None),
             lambda: mfr.nvfp4_quantize(x, torch.ones(2).cuda()), lambda: mfr.nvfp4_quantize(x, s, codes=u8(4, 31)),
             lambda: mfr.nvfp4_quantize(x, s, sf=u8(4, 5)), lambda: mfr.nvfp4_dequantize(u8(4, 32), u8(4, 3), s),
             lambda: mfr.moe_expert_matmul_nvfp4(u8(4, 32), u8(4, 4), u8(2, 128, 32), u8(2, 511), o),
             lambda: mfr.moe_expert_matmul_nvfp4(u8(4, 32), u8(4, 4), u8(2, 128, 32), u8(2, 512), o, alpha=s)]
    for call in wrong:
        with pytest.raises(ValueError):
            call()
    refused = [lambda: mfr.moe_expert_matmul(x[:, :60], w[:, :, :60], o), lambda: mfr.moe_expert_matmul(x, w[:, :12], o),
               lambda: mfr.moe_expert_matmul(x.expand(4, 64)[:1].expand(4, 64), w, o),  # (rows that are one row)
               lambda: mfr.moe_expert_matmul(x, w, o, gate_up=d),
               lambda: mfr.moe_expert_matmul_backward(d, x, w, o, d_weight=w.clone(), accumulate=True),
               lambda: mfr.nvfp4_quantize(x[:, :24].contiguous(), s),
               lambda: mfr.moe_expert_matmul_nvfp4(u8(4, 48), u8(4, 6), u8(2, 128, 48), u8(2, 1024), o),
               lambda: mfr.moe_expert_matmul_nvfp4(u8(4, 32), u8(4, 4), u8(2, 128, 32), u8(2, 512), o, gated=True)]
    for call in refused:
        with pytest.raises(mfr.MoEFinalizeError):
            call()
    torch.cuda.synchronize()


def _nvfp4_large(seed):
    """A case whose rows' scales take the workspace, and its result."""
    g = torch.Generator().manual_seed(seed)
    counts, n_in, n = [130, 0, 250, 41], 320, 136
    off, R = ref.order(counts)
    codes, wc = (torch.randint(0, 256, s, generator=g, dtype=torch.uint8) for s in ((R, n_in // 2), (4, n, n_in // 2)))
    sf, ws = (torch.randint(40, 60, s, generator=g, dtype=torch.uint8) for s in ((R, n_in // 16), (4, 256 * (n_in // 16))))
    return [t.cuda() for t in (codes, sf, wc, ws, off, torch.tensor(counts, dtype=torch.int32))]


def test_nvfp4_on_other_streams_and_without_programmatic_launch(mfr):
    args = _nvfp4_large(1)
    assert mfr.moe_expert_matmul_nvfp4_workspace_bytes(4, args[0].shape[0], 320) > 0
    want = mfr.moe_expert_matmul_nvfp4(*args, pdl=False)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [mfr.moe_expert_matmul_nvfp4(*args, stream=streams[i % 2], pdl=i % 3 > 0) for i in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    x, w, d, off, cnt = (t.cuda() for t in _case([300, 5, 0, 250], 136, 264, 2))
    for call in (lambda p: mfr.moe_expert_matmul(x, w, off, cnt, pdl=p), lambda p: mfr.moe_expert_matmul_backward(d, x, w, off, cnt, pdl=p)[0],
                 lambda p: mfr.moe_swiglu_backward(x[:, :64], d[:, :128], pdl=p)[0], lambda p: mfr.nvfp4_quantize(d[:, :256], torch.ones(1).cuda(), pdl=p)[0]):
        assert torch.equal(call(True), call(False))


def test_two_graphs_at_once(mfr):
    """Two captured graphs, each with the workspace that its call allocated, replayed beside each other."""
    cases = [_nvfp4_large(s) for s in (3, 4)]
    wants = [mfr.moe_expert_matmul_nvfp4(*c) for c in cases]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for c, s in zip(cases, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append([mfr.moe_expert_matmul_nvfp4(*c) for _ in range(3)])
        graphs.append(g)
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for held, w in zip(outs, wants) for o in held)


def test_a_workspace_that_is_passed_in(mfr):
    args = _nvfp4_large(5)
    need = mfr.moe_expert_matmul_nvfp4_workspace_bytes(4, args[0].shape[0], 320)
    space = torch.full((need + 512,), 0x7f, dtype=torch.uint8).cuda()  # scales that are not numbers, where it is not written
    assert torch.equal(mfr.moe_expert_matmul_nvfp4(*args, workspace=space), mfr.moe_expert_matmul_nvfp4(*args))
    assert (space[need:] == 0x7f).all()
    with pytest.raises(mfr.MoEFinalizeError):
        mfr.moe_expert_matmul_nvfp4(*args, workspace=space[:need - 1])
    with pytest.raises(ValueError):
        mfr.moe_expert_matmul_nvfp4(*args, workspace=space.cpu())


@pytest.mark.parametrize("rows", [3, 700])
@pytest.mark.parametrize("call", ["product", "rows", "weights", "nvfp4"])
def test_a_wait_that_runs_out_is_counted(mfr, call, rows):
    """A barrier that expects one arrival more than come: the call ends after its limit, is counted, and the next one is right."""
    X, timeout = mfr.experts, mfr.MFR_FLAG_TEST_STREAM_TIMEOUT
    x, w, d, off, cnt = (t.cuda() for t in _case([rows], 128, 256, 20))
    dx, dw, out = torch.empty_like(x), torch.empty_like(w), torch.empty_like(d)
    ptr = lambda *ts: [t.data_ptr() for t in ts]  # noqa: E731
    codes, wc, ws = (torch.zeros(*s, dtype=torch.uint8).cuda() for s in ((rows, 64), (1, 256, 64), (1, 256 * 8)))
    sf, space = torch.zeros(rows, 8, dtype=torch.uint8).cuda(), torch.zeros(1 << 20, dtype=torch.uint8).cuda()
    if call == "product":
        f, args = "moe_expert_matmul", X._pack_matmul(1, 128, 256, 1, 0, rows, x.data_ptr(), 128, w.data_ptr(), 128, 256 * 128, *ptr(off, cnt, out), 256, 0, 0, timeout)
    elif call == "nvfp4":
        f, args = "moe_expert_matmul_nvfp4", X._pack_matmul_nvfp4(1, 128, 256, 1, 0, rows, *ptr(codes, sf, wc, ws), 0, *ptr(off, cnt, out), 256, space.data_ptr(), 1 << 20, timeout)
    else:
        f, args = "moe_expert_matmul_backward", X._pack_matmul_backward(
            1, 128, 256, 1, 1, 0, rows, x.data_ptr(), 128, w.data_ptr(), 128, 256 * 128, d.data_ptr(), 256, *ptr(off, cnt),
            dx.data_ptr() if call == "rows" else 0, 128, dw.data_ptr() if call == "weights" else 0, timeout)
    assert mfr.moe_expert_read_timeouts() == 0
    assert getattr(mfr.raw_library(), f)(args, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert mfr.moe_expert_read_timeouts() > 0 and mfr.moe_expert_read_timeouts() == 0
    assert torch.equal(mfr.moe_expert_matmul(x, w, off, cnt).cpu(), _want(x.cpu(), w.cpu(), off.cpu(), [rows]).half())
    got = mfr.moe_expert_matmul_backward(d, x, w, off, cnt)
    assert torch.equal(got[0].cpu(), (d.double() @ w[0].double()).half().cpu()) and torch.equal(got[1][0].cpu(), (d.double().T @ x.double()).half().cpu())
    assert mfr.moe_expert_read_timeouts() == 0
