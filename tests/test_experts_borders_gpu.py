"""The experts' products where they can go wrong: gates far below zero, as many rows as a call takes, experts that share
rows, reductions longer than a wait, waits on other streams."""
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


# ----------------------------------------------------------------------------------------------------------------
# The gate
# ----------------------------------------------------------------------------------------------------------------

def _spread(g, *shape):
    """BF16 values of either sign over most of the type's range."""
    sign = 1.0 - 2.0 * torch.randint(0, 2, shape, generator=g)
    return (sign * torch.exp((torch.rand(*shape, generator=g) * 2 - 1) * 86)).to(BF)


def _gates(g, *shape):
    """Gates whose exponential halves stay normal numbers in FP32, most of them below zero."""
    return (torch.rand(*shape, generator=g) * 200 - 168).to(BF)


def _near(name, got, want, rel):
    """One rounding to BF16 of a value that is off by at most ``rel`` of it, below the type's normal numbers by one of them, and
    infinite where the value may round beyond the largest."""
    got, off, tiny = got.double(), rel * want.abs(), 2.0 ** -126
    top = torch.finfo(BF).max
    beyond = want.abs() + off > top
    assert (torch.isfinite(got) | beyond).all(), f"{name} is not finite"
    assert ((got == torch.sign(want) * float("inf")) | ((got - want).abs() <= off + 2.0 ** -8 * (want.abs() + off)) | ~beyond).all(), name
    bad = ~beyond & ((got - want).abs() > off + 2.0 ** -8 * (want.abs() + off) + tiny)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off"


def _logistic(g):
    return torch.where(g >= 0, 1 / (1 + torch.exp(-g)), torch.exp(g) / (1 + torch.exp(g)))


@pytest.mark.parametrize("rows", [8, 64])
def test_the_gate_of_large_negative_values(mfr, rows):
    """Rows with a single one pick out the weights, so the gate's inputs are the weights' BF16 values: its output is g / (1 + exp(-g)) * u
    wherever that is a normal number, however small the quotient alone is."""
    F, n_in = 128, 64
    g = torch.Generator().manual_seed(rows)
    gate, up = _gates(g, F, n_in), _spread(g, F, n_in)
    gate[0, :8] = torch.tensor([-87.0, -87.5, -88.0, -88.5, -89.0, -95.0, -104.0, -1e4]).to(BF)
    up[0, :8] = torch.tensor([1e33, 1e33, 1e33, 1e33, 1e35, 1e38, 1e38, 1e38]).to(BF)
    x = torch.eye(n_in)[torch.arange(rows) % n_in].to(BF)
    off, cnt = torch.tensor([0, rows], dtype=torch.int32).cuda(), torch.tensor([rows], dtype=torch.int32).cuda()
    out = mfr.moe_expert_matmul(x.cuda(), torch.cat([gate, up])[None].cuda(), off, cnt, gated=True).cpu()
    a, b = gate.double().T[:rows], up.double().T[:rows]
    # the exponential of half the gate, twice: 2^-22 each, and 0.75 |g| * 2^-23 by the rounding of its argument; a few operations
    _near("out", out, a * _logistic(a) * b, (a.abs() + 8) * 2.0 ** -23)


def test_gates_below_the_border_leave_their_neighbours_alone(mfr):
    """A row's results are the same beside rows with gates far below zero."""
    g = torch.Generator().manual_seed(5)
    x, w = torch.randn(64, 64, generator=g).to(BF), torch.randn(1, 256, 64, generator=g).to(BF)
    off, cnt = torch.tensor([0, 64], dtype=torch.int32).cuda(), torch.tensor([64], dtype=torch.int32).cuda()
    plain = mfr.moe_expert_matmul(x.cuda(), w.cuda(), off, cnt, gated=True)
    beside = x.clone()
    beside[::2] = 100 * x[::2]  # gates of either sign, to -3000
    out = mfr.moe_expert_matmul(beside.cuda(), w.cuda(), off, cnt, gated=True)
    assert torch.equal(out[1::2], plain[1::2]) and (x[::2].float() @ w[0, :128].float().T * 100).min() < -1000


def test_the_gates_gradient_of_large_negative_values(mfr):
    R, F = 40, 512
    g = torch.Generator().manual_seed(3)
    gate, up, d = _gates(g, R, F), _spread(g, R, F), _spread(g, R, F)
    gate[0, :8] = torch.tensor([-87.5, -88.5, -89.0, -95.0, -115.0, -60.0, -1e4, -150.0]).to(BF)
    up[0, :8] = torch.tensor([1e33, 1e33, 1e35, 1e38, 3e38, 1e20, 1e38, 1e37]).to(BF)
    d[0, :8] = torch.tensor([1.0, 1.0, 1e-3, 1e10, 1e-25, 1e20, 1e38, 1e37]).to(BF)
    d_x, y = (t.cpu() for t in mfr.moe_swiglu_backward(d.cuda(), torch.cat([gate, up], 1).cuda()))
    a, b, e = gate.double(), up.double(), d.double()
    p, rel = _logistic(a), (a.abs() + 8) * 2.0 ** -23
    _near("act", y, a * p * b, rel)
    _near("d_up", d_x[:, F:], e * a * p, rel)
    # 1 + g (1 - p) has a zero; its error is relative to its terms
    slope = 1 + a * (1 - p)
    _near("d_gate", d_x[:, :F], e * b * p * slope, rel * (1 + 2 * a.abs()) / slope.abs())


# ----------------------------------------------------------------------------------------------------------------
# Rows
# ----------------------------------------------------------------------------------------------------------------

def _room(gb):
    """Skips where so many GB are not free."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"{gb} GB of device memory are wanted")


def _count(t):
    """Elements that are not zero, a piece at a time."""
    return sum(int(torch.count_nonzero(p)) for p in t.split(1 << 27))


def test_the_most_rows_there_may_be(mfr):
    """One expert of as many rows as a call takes: the first, the last and some between hold values, the others zeros."""
    R, n = (1 << 31) - 1024, 8
    _room(90)
    g = torch.Generator().manual_seed(4)
    at = torch.cat([torch.arange(300), torch.randint(300, R - 300, (400,), generator=g).unique(), torch.arange(R - 300, R)]).cuda()
    x, y = torch.zeros(R, n, dtype=HF, device="cuda"), torch.empty(R, n, dtype=HF, device="cuda")
    some, w = torch.randint(1, 3, (at.numel(), n), generator=g).to(HF).cuda(), torch.randint(1, 3, (1, n, n), generator=g).to(HF).cuda()
    x[at] = some
    off, cnt = torch.tensor([0, R], dtype=torch.int32).cuda(), torch.tensor([R], dtype=torch.int32).cuda()
    for product, want in ((lambda: mfr.moe_expert_matmul(x, w, off, cnt, out=y), some.double() @ w[0].double().T),
                          (lambda: mfr.moe_expert_matmul_backward(x, None, w, off, cnt, d_rows=y, want_d_weight=False), some.double() @ w[0].double())):
        y.fill_(1.0)
        product()
        assert torch.equal(y[at].double(), want) and _count(y) == want.numel()


def test_experts_that_share_all_rows_end(mfr):
    """Offsets that give every expert every row: the tiles that 1024 experts would fill pass 2^32, those that the call works on are
    no more than its rows fill."""
    E, R, n = 1024, 1 << 29, 8
    _room(40)
    off, cnt = torch.zeros(E + 1, dtype=torch.int32).cuda(), torch.full((E,), R, dtype=torch.int32).cuda()
    x, y = torch.zeros(R, n, dtype=HF, device="cuda"), torch.full((R + 1, n), 7.0, dtype=HF, device="cuda")
    w = torch.ones(E, n, n, dtype=HF).cuda()
    mfr.moe_expert_matmul(x, w, off, cnt, out=y[:R])
    mfr.moe_expert_matmul_backward(x, None, w, off, cnt, d_rows=y[:R], want_d_weight=False)
    assert (y[R] == 7).all() and mfr.moe_expert_read_timeouts() == 0
    del x, y
    R = 1 << 25
    cnt.fill_(R)
    codes, sf = torch.zeros(R, 32, dtype=torch.uint8, device="cuda"), torch.zeros(R, 4, dtype=torch.uint8, device="cuda")
    y = torch.full((R + 1, n), 7.0, dtype=BF, device="cuda")
    space = torch.full((mfr.moe_expert_matmul_nvfp4_workspace_bytes(E, R, 64) + 4096,), 9, dtype=torch.uint8, device="cuda")
    mfr.moe_expert_matmul_nvfp4(codes, sf, torch.zeros(E, n, 32, dtype=torch.uint8).cuda(), torch.zeros(E, 512, dtype=torch.uint8).cuda(), off, cnt,
                                out=y[:R], workspace=space)
    assert (y[R] == 7).all() and (space[-4096:] == 9).all() and mfr.moe_expert_read_timeouts() == 0


@pytest.mark.parametrize("n_out", [8, 136])
def test_a_reduction_that_takes_longer_than_a_wait(mfr, n_out):
    """The weights' gradient of an expert of so many rows is at work on one tile for more than the 2 s of a wait (64 rows are four
    instructions of at least 128 cycles each), by one CTA and by a pair."""
    R, n_in = 640_000_001, 8
    _room(20 + R * (n_in + n_out) * 2 // (1 << 30))
    g = torch.Generator().manual_seed(n_out)
    at = torch.cat([torch.arange(100), torch.randint(100, R - 100, (300,), generator=g).unique(), torch.arange(R - 100, R)]).cuda()
    x, d = torch.zeros(R, n_in, dtype=HF, device="cuda"), torch.zeros(R, n_out, dtype=HF, device="cuda")
    some, grad = torch.randint(-2, 3, (at.numel(), n_in), generator=g).to(HF).cuda(), torch.randint(-2, 3, (at.numel(), n_out), generator=g).to(HF).cuda()
    x[at], d[at] = some, grad
    off, cnt = torch.tensor([0, R], dtype=torch.int32).cuda(), torch.tensor([R], dtype=torch.int32).cuda()
    _, dw = mfr.moe_expert_matmul_backward(d, x, None, off, cnt, want_d_rows=False, d_weight_dtype=F32)
    torch.cuda.synchronize()
    assert mfr.moe_expert_read_timeouts() == 0
    assert torch.equal(dw[0].double(), grad.double().T @ some.double())


# ----------------------------------------------------------------------------------------------------------------
# Waits
# ----------------------------------------------------------------------------------------------------------------

def test_a_wait_that_runs_out_on_another_stream_is_counted(mfr):
    """The count waits for every stream of the device: the call may still be running."""
    X, rows = mfr.experts, 40
    x, w = torch.ones(rows, 64, dtype=HF).cuda(), torch.ones(1, 64, 64, dtype=HF).cuda()
    off, cnt, out = torch.tensor([0, rows], dtype=torch.int32).cuda(), torch.tensor([rows], dtype=torch.int32).cuda(), torch.empty(rows, 64, dtype=HF).cuda()
    args = X._pack_matmul(1, 64, 64, 1, 0, rows, x.data_ptr(), 64, w.data_ptr(), 64, 64 * 64, off.data_ptr(), cnt.data_ptr(), out.data_ptr(), 64, 0, 0,
                          mfr.MFR_FLAG_TEST_STREAM_TIMEOUT)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert mfr.moe_expert_read_timeouts() == 0
    assert mfr.raw_library().moe_expert_matmul(args, side.cuda_stream) == 0
    first = mfr.moe_expert_read_timeouts()
    torch.cuda.synchronize()
    again = mfr.moe_expert_read_timeouts()
    assert first > 0 and again == 0
    assert torch.equal(mfr.moe_expert_matmul(x, w, off, cnt), torch.full((rows, 64), 64.0, dtype=HF).cuda())


# ----------------------------------------------------------------------------------------------------------------
# Refusals
# ----------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("no_tensor", [3, [1.0], "rows"])
def test_what_is_no_tensor_is_refused(mfr, no_tensor):
    x, w, o = torch.zeros(4, 64, dtype=BF).cuda(), torch.zeros(2, 128, 64, dtype=BF).cuda(), torch.zeros(3, dtype=torch.int32).cuda()
    d = torch.zeros(4, 128, dtype=BF).cuda()
    t = no_tensor
    for call in (lambda: mfr.moe_expert_matmul(x, w, o, out=t), lambda: mfr.moe_expert_matmul(x, w, o, gated=True, gate_up=t),
                 lambda: mfr.moe_expert_matmul(x, w, t), lambda: mfr.moe_expert_matmul(x, w, o, t),
                 lambda: mfr.moe_expert_matmul_backward(d, x, w, t), lambda: mfr.moe_expert_matmul_backward(d, x, w, o, t),
                 lambda: mfr.moe_expert_matmul_backward(d, x, w, o[0]), lambda: mfr.moe_expert_matmul_backward(d, t, w, o),
                 lambda: mfr.moe_expert_matmul_backward(d, x, w, o, d_rows=t), lambda: mfr.moe_expert_matmul_backward(d, x, w, o, d_weight=t),
                 lambda: mfr.moe_swiglu_backward(t, d), lambda: mfr.moe_swiglu_backward(x, d, d_gate_up=t),
                 lambda: mfr.moe_swiglu_backward(x, d, act=t), lambda: mfr.moe_swiglu_backward(x, d, row_route=t),
                 lambda: mfr.nvfp4_quantize(x, t), lambda: mfr.nvfp4_quantize(x, d, codes=t)):
        with pytest.raises(ValueError):
            call()
