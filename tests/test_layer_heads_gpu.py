"""The head norm with rotation where a value is not finite or a position is far."""
import pytest
import torch

import layer_reference as ref
from layer_reference import smallest, step

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def mfr():
    import moe_finalize_residual_gb300 as m
    return m


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


PARTLY = [(64, 32, "half"), (64, 16, "half"), (64, 48, "half"), (48, 0, "half"), (80, 30, "interleaved"), (64, 6, "interleaved"),
          (32, 16, "interleaved"), (16, 0, "interleaved"), (512, 256, "half"), (128, 126, "interleaved")]


@pytest.mark.parametrize("D,rot,style", PARTLY)
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float16])
def test_an_infinity_stays_out_of_unrotated_elements(mfr, D, rot, style, act):
    """Head h of the queries has an infinity in its unrotated element rot + h.  Its root mean square is infinite, so by the
    formula every finite element that passes is zero and the infinite one NaN; whatever shares a lane with it."""
    heads = D - rot
    q = torch.randn(2, heads, D, generator=gen(D)).to(act)
    at = rot + torch.arange(heads)
    q[0, torch.arange(heads), at] = torch.where(torch.arange(heads) % 2 == 0, INF, -INF).to(act)
    k = torch.randn(2, 3, D, generator=gen(1)).to(act)
    w = (1 + 0.1 * torch.randn(D, generator=gen(2))).to(act).cuda()
    pos, freq = torch.tensor([5, 7]).cuda(), torch.rand(rot // 2, generator=gen(3)).cuda()
    y, yk = mfr.head_norm_rotary(q.cuda(), k.cuda(), w, w, pos, freq, style=style)
    y = y.cpu()
    hit = torch.zeros(heads, D, dtype=torch.bool)
    hit[torch.arange(heads), at] = True
    assert torch.isnan(y[0][hit]).all()
    assert (y[0][~hit] == 0).all(), f"{int((~(y[0] == 0) & ~hit).sum())} of {heads * (D - 1)} finite elements are not 0"
    clean, clean_k = mfr.head_norm_rotary(torch.nan_to_num(q, posinf=1.0, neginf=1.0).cuda(), k.cuda(), w, w, pos, freq, style=style)
    assert torch.equal(y[1], clean[1].cpu()) and torch.equal(yk, clean_k)


@pytest.mark.parametrize("D,rot,style", PARTLY)
@pytest.mark.parametrize("bad", [INF, float("nan")])
def test_a_weight_stays_out_of_unrotated_elements(mfr, D, rot, style, bad):
    q = torch.randn(3, 2, D, generator=gen(D)).half().cuda()
    pos, freq = torch.tensor([0, 1, 9]).cuda(), torch.rand(rot // 2, generator=gen(3)).cuda()
    good = torch.ones(D, dtype=torch.float16).cuda()
    want, _ = mfr.head_norm_rotary(q, q, good, good, pos, freq, style=style)
    for i in range(rot, D, max(1, (D - rot) // 24)):
        w = good.clone()
        w[i] = bad
        y, _ = mfr.head_norm_rotary(q, q, w, good, pos, freq, style=style)
        keep = torch.arange(D) != i
        assert torch.equal(y[:, :, keep], want[:, :, keep]) and not torch.isfinite(y[:, :, i]).any(), i


@pytest.mark.parametrize("D,rot,style", PARTLY)
@pytest.mark.parametrize("bad", [INF, float("nan")])
def test_a_gradient_stays_out_of_unrotated_weights(mfr, D, rot, style, bad):
    """d_out of one unrotated element is not finite: of the weights' gradients only its own takes that up."""
    g = gen(D)
    q = (0.5 + torch.rand(3, 2, D, generator=g)).half().cuda()
    d = torch.randn(3, 2, D, generator=g).half().cuda()
    w = torch.ones(D, dtype=torch.float16).cuda()
    pos, freq = torch.tensor([0, 1, 9]).cuda(), torch.rand(rot // 2, generator=gen(3)).cuda()
    want = mfr.head_norm_rotary_backward(d, d, q, q, w, w, pos, freq, style=style)
    for i in range(rot, D, max(1, (D - rot) // 24)):
        hit = d.clone()
        hit[1, 1, i] = bad
        got = mfr.head_norm_rotary_backward(hit, d, q, q, w, w, pos, freq, style=style)
        keep = (torch.arange(D) != i).cuda()
        assert torch.equal(got[2][keep], want[2][keep]) and not torch.isfinite(got[2][i]), i
        assert torch.equal(got[3], want[3]) and torch.equal(got[0][0], want[0][0]) and torch.equal(got[0][1, 0], want[0][1, 0])


# As a share of its pair's length, before the rounding: the mean square 15 u, half of it in the root, and the root 4 u; the
# element times the root u; the angle pi 2^-25 (the nearest 2^-32 turn, and the half turn's rounding) and 2^-47 of a turn;
# the sine or cosine 2 u, times rotary_scale u, times the weight u; the products and their sum 2 u on both elements.
U = 2.0 ** -24
SHARE = 22 * U + 1.2e-7 + 2.0 ** -44


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("wide", [False, True])
def test_far_positions_lose_nothing(mfr, style, act, wide):
    """Every position that its type holds, and frequencies up to the largest allowed, forward and back."""
    D = 64
    pos = [0, 1, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1] + [2 ** 33 + 5, 2 ** 39 + 3, 10 ** 13 + 9, 10 ** 15 + 7, 2 ** 53 + 1, 2 ** 62 - 3,
                                                              2 ** 63 - 1] * wide
    freq = torch.cat([torch.tensor([1.0, 0.5, 3.25, -0.7, 0.0, 900.0, 1e-9, -1e-18, 3e-39, 60000.5, 1048575.9, -777777.7]),
                      torch.rand(D // 2 - 12, generator=gen(1))])
    x = torch.randn(len(pos), 2, D, generator=gen(2)).to(act)
    d = torch.randn(len(pos), 2, D, generator=gen(3)).to(act)
    at = torch.tensor(pos, dtype=torch.int64 if wide else torch.int32).cuda()
    y, _ = mfr.head_norm_rotary(x.cuda(), x.cuda(), None, None, at, freq.cuda(), style=style, eps=1e-5)
    x64 = x.double().requires_grad_()
    want = ref.head_norm(x64, None, pos, freq, style, 1e-5, 1.0)
    r = 1 / (x.double().pow(2).mean(2, keepdim=True) + 1e-5).sqrt()

    def pair_size(v):
        a, b = (v[..., :D // 2], v[..., D // 2:]) if style == "half" else (v[..., 0::2], v[..., 1::2])
        n = torch.hypot(a, b)
        return torch.cat([n, n], 2) if style == "half" else n.repeat_interleave(2, dim=2)

    def close(got, want, before):
        bound = before + step(act) * (want.abs() + before) + smallest(act)
        bad = (got.double().cpu() - want).abs() > bound
        assert not bad.any(), f"positions {[pos[i] for i in bad.any(2).any(1).nonzero().flatten()]}"

    close(y, want.detach(), SHARE * pair_size((x.double() * r)))
    (want * d.double()).sum().backward()
    dx = mfr.head_norm_rotary_backward(d.cuda(), d.cuda(), x.cuda(), x.cuda(), None, None, at, freq.cuda(), style=style, eps=1e-5)[0]
    # r (g - x r^2 mean(g x)): the share on every factor, and the mean's 21 additions on its terms
    size = pair_size(d.double())
    mean = (size * x.double().abs()).mean(2, keepdim=True)
    close(dx, x64.grad, r * (2 * SHARE * size + x.double().abs() * r * r * mean * (3 * SHARE + 24 * U)))
