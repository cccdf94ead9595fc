"""The operators around the finalize where a decision between experts is close."""
import numpy as np
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu

FLOAT_MAX = torch.finfo(torch.float32).max


@pytest.fixture(scope="module")
def mfr():
    import moe_finalize_residual_gb300 as m
    return m


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def wrong_tokens(mfr, x, K, score, bias, G=1, Gk=1, top2=False):
    """How many tokens get other ids than the definition in 64 bits gives."""
    got = mfr.moe_route(x.cuda(), K, score=score, bias=bias.cuda(), num_groups=G, topk_groups=Gk,
                        group_score="top2" if top2 else "max", order=False).expert_ids.cpu().numpy()
    want = ref.choose(x.double().numpy(), K, score, bias.double().numpy(), G, Gk, top2)[0]
    return int((got != want).any(1).sum())


def graph_time(f, launches=10):
    """Median time of a call in a graph of them, in us."""
    f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(launches):
            f()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    times = []
    for _ in range(13):
        start.record()
        g.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 1e3 / launches)
    return sorted(times[3:])[5]


# ------------------------------------------------------------------------------------------------------------
# Choices that are close
# ------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_is_not_decided_again_where_few_lanes_hold_an_expert(mfr, score):
    """Two of eight groups leave fewer lanes with experts than places; random scores are as far apart as with four, so
    no more tokens may need 64 bits.  (All of them did: 4 to 9 times the time; now 1.4.)"""
    x, bias = torch.randn(16384, 256, generator=gen(0)).cuda(), 0.05 * torch.randn(256, generator=gen(1)).cuda()
    two, four = (graph_time(lambda: mfr.moe_route(x, 8, score=score, bias=bias, num_groups=8, topk_groups=n,
                                                  group_score="top2", order=False)) for n in (2, 4))
    assert two < 2.5 * four, f"{two:.1f} us with 2 groups kept, {four:.1f} with 4"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [24, 32, 64, 128, 256, 512, 896])
@pytest.mark.parametrize("level", [0.0, 1.0, 0.5, -0.25])
def test_route_scores_near_one_another_without_groups(mfr, score, E, level):
    """Biases that level a token's scores to within an FP32 rounding: the candidates' cut must not lose an expert that
    64 bits put first.  Token 0 of each draw is level (1.0 stands for 1 / E), token 1 is not."""
    level = 1.0 / E if level == 1.0 else level
    wrong = {}
    for seed in range(12):
        x = torch.randn(2, E, generator=gen(100 * E + seed))
        s = ref.choose(x[:1].double().numpy(), 1, score)[1][0]
        bias = torch.from_numpy(level - s).float()
        for K in (1, 2, 8, 22, 33):
            if K <= E:
                n = wrong_tokens(mfr, x, K, score, bias)
                wrong[K] = wrong.get(K, 0) + n
    assert not any(wrong.values()), f"tokens with other ids, by K: {wrong}"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(64, 4), (256, 8), (512, 8), (900, 4), (96, 3)])
@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("level", [0.0, 0.5])
def test_route_scores_near_one_another_in_groups(mfr, score, E, G, top2, level):
    wrong = {}
    for seed in range(6):
        x = torch.randn(2, E, generator=gen(7 * E + seed))
        s = ref.choose(x[:1].double().numpy(), 1, score)[1][0]
        bias = torch.from_numpy(level - s).float()
        bias[: E // 2] += 0.125 * (seed % 2)  # every other draw: the groups' border lies elsewhere than the experts'
        for K, Gk in ((2, 1), (8, 2), (8, G - 1), (20, G)):
            n = wrong_tokens(mfr, x, K, score, bias, G, Gk, top2)
            wrong[K, Gk] = wrong.get((K, Gk), 0) + n
    assert not any(wrong.values()), f"tokens with other ids, by K and kept groups: {wrong}"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,few", [(256, 40), (512, 70), (1024, 90), (128, 30)])
def test_route_few_near_scores_among_many(mfr, score, E, few):
    """Only some experts are level; they lie in few lanes, so that the lanes' best say little about the cut."""
    wrong = {}
    for seed in range(8):
        x = torch.randn(2, E, generator=gen(E + seed))
        s = ref.choose(x[:1].double().numpy(), 1, score)[1][0]
        bias = torch.from_numpy(-1.0 - s).float()
        bias[:few] += 1.25
        bias[few: 2 * few: 2] += 1.25 + 2.0 ** -20 * torch.arange(len(bias[few: 2 * few: 2])).float() / few
        for K in (2, 8, 20, 40):
            n = wrong_tokens(mfr, x, K, score, bias)
            wrong[K] = wrong.get(K, 0) + n
    assert not any(wrong.values()), f"tokens with other ids, by K: {wrong}"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [8.0, 1000.0, 30000.0])
@pytest.mark.parametrize("E,G,Gk,K", [(64, 32, 16, 8), (16, 8, 3, 2), (96, 32, 5, 4), (512, 16, 4, 8), (600, 24, 7, 6)])
def test_route_group_sums_that_cancel(mfr, score, size, E, G, Gk, K):
    """A group's two best scores near +size and -size: their sum is small, the roundings of the two are not."""
    wrong = 0
    for seed in range(20):
        g = gen(E + seed)
        x = torch.randn(3, E, generator=g)
        s = ref.choose(x[:1].double().numpy(), 1, score)[1][0].reshape(G, E // G)
        bias = np.full((G, E // G), -10.0 * size)  # the third and later ones of a group do not count
        bias[:, 0] = size * (1 + torch.rand(G, generator=g).double().numpy() / 16)
        bias[:, 0] = np.float32(bias[:, 0])
        bias[:, 1] = 0.25 - s[:, 0] - s[:, 1] - bias[:, 0]  # level sums, to half a step of the second bias
        wrong += wrong_tokens(mfr, x, K, score, torch.from_numpy(bias.reshape(-1)).float(), G, Gk, True)
    assert wrong == 0, f"{wrong} of 60 tokens got other ids"


def test_route_random_groups_of_two_whose_scores_cancel(mfr):
    x = torch.randn(50000, 16, generator=gen(3))
    bias = torch.tensor([1000.0, -1000.0]).repeat(8) + 0.1 * torch.randn(16, generator=gen(4))
    assert wrong_tokens(mfr, x, 2, "sigmoid", bias, 8, 3, True) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,Gk,K", [(64, 8, 4, 8), (64, 8, 8, 40), (60, 4, 2, 10), (256, 8, 4, 8), (200, 8, 3, 60)])
@pytest.mark.parametrize("end", [-1.0, 1.0])
@pytest.mark.parametrize("top2", [False, True])
def test_route_group_sums_past_the_largest_number(mfr, score, E, G, Gk, K, end, top2):
    """Biases at either end of FP32 on some groups, as masks use them: a sum of two is finite in 64 bits."""
    wrong = 0
    for seed in range(8):
        g = gen(E + seed)
        x = torch.randn(20, E, generator=g)
        bias = 0.1 * torch.randn(E, generator=g)
        off = torch.rand(E, generator=g) < 0.3
        off.view(G, E // G)[torch.randperm(G, generator=g)[: G - (seed % 3)]] = True  # all groups but 0, 1 or 2
        bias[off] = end * FLOAT_MAX
        bias[off & (torch.rand(E, generator=g) < 0.5)] = end * FLOAT_MAX * 0.75
        wrong += wrong_tokens(mfr, x, K, score, bias, G, Gk, top2)
    assert wrong == 0, f"{wrong} of 160 tokens got other ids"
