"""Edges of the scored router on the GPU: scores that only a division makes equal, weights at the end of f32, streams."""
import numpy as np
import pytest

from oracle import scored

pytestmark = pytest.mark.gpu


def _route(lg, k, **rule):
    import torch
    import nvfp4_weight_only_top_b200 as moe
    if rule.get("bias") is not None:
        rule["bias"] = torch.from_numpy(rule["bias"]).cuda()
    r = moe.moe_nvfp4_route_scored(torch.from_numpy(lg).cuda(), moe.make_router(**rule), k)
    torch.cuda.synchronize()
    return {n: v.cpu().numpy() for n, v in r.items()}


def test_softmax_scores_that_the_division_makes_equal():
    """exp(-2^-53) and exp(0) divided by this row's sum are one double: the lower index of the two comes first."""
    lg = np.full((1, 9), -1.0, dtype=np.float32)
    lg[0, 5], lg[0, 1], lg[0, 0] = 0.0, -2.0 ** -53, -2.0 ** -52
    ids, _ = scored.route_scored(lg, 3, score="softmax")
    assert ids.tolist() == [[1, 5, 0]]
    assert _route(lg, 3, score="softmax")["ids"].tolist() == [[1, 5, 0]]


@pytest.mark.parametrize("T", [6, 900])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_a_bias_of_zeros_changes_nothing(T, groups, top_groups, group_top):
    """Softmax scores whose exponentials lie a few steps of 64 bits apart: without a bias the order is found from the
    exponentials, with one from the quotients."""
    rng = np.random.default_rng(T + group_top)
    lg = np.empty((T, 64), dtype=np.float32)
    for t in range(T):
        lg[t] = rng.choice([-1.0, -2.0, -3.5, -np.inf], 64)
        lg[t, rng.choice(64, 9, replace=False)] = -(rng.integers(0, 6, 9) * 2.0 ** -53)
    rule = dict(score="softmax", groups=groups, top_groups=top_groups, group_top=group_top)
    for x in (lg, rng.integers(-3, 4, (T, 64)).astype(np.float32)):
        a = _route(x, 6, **rule)
        b = _route(x, 6, bias=np.zeros(64, dtype=np.float32), **rule)
        assert all(np.array_equal(a[n], b[n]) for n in a if n != "w")
        # weights of two ways: two exponentials (2 steps each), a sum, a division, a tree of 5 additions and a division
        # in 32 bits on one side and 64 bits rounded once on the other, under 16 half steps of 2^-24
        assert (np.abs(a["w"] - b["w"]) <= 16 * 2.0 ** -24 * np.abs(b["w"])).all()


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_small_weights(score, renormalize):
    """Chosen experts whose scores are at the end of f32, with a scale that takes them back into its range.

    Error: 16 half steps of 2^-24 (two exponentials, a sum, a division, a tree of additions, a division, the scale),
    and the rounding of an exponent's argument, up to 48 x 2^-24 for a softmax's; 2^-149 where the weight is subnormal."""
    rng = np.random.default_rng(17)
    T, E, k = 40, 32, 6
    far = np.exp2(rng.uniform(3, 9.4, (T, 1)))                   # 8 .. 676 below the largest
    lg = -(far + 8 * rng.random((T, E))).astype(np.float32)
    if score == "softmax":
        lg[:, 7] = rng.standard_normal(T)
        lg += 3 * rng.standard_normal((T, 1)).astype(np.float32)
    lg = lg.astype(np.float32)
    for scale in (1.0, 2.0 ** 60, 2.0 ** 120):
        w = _route(lg, k, score=score, renormalize=renormalize, scale=scale)["w"]
        ids, want = scored.route_scored(lg, k, score=score, renormalize=renormalize, scale=scale)
        assert (np.abs(w - want) <= 64 * 2.0 ** -24 * want + 2.0 ** -149).all(), scale


def test_a_bias_whose_storage_changes():
    """The router reads the bias tensor as it is at the call."""
    import torch
    import nvfp4_weight_only_top_b200 as moe
    lg = torch.zeros(3, 16, device="cuda")
    bias = torch.zeros(16, device="cuda")
    router = moe.make_router(bias=bias)
    assert moe.moe_nvfp4_route_scored(lg, router, 2)["ids"].tolist() == [[0, 1]] * 3
    bias.data = torch.arange(16, dtype=torch.float32, device="cuda")
    assert moe.moe_nvfp4_route_scored(lg, router, 2)["ids"].tolist() == [[15, 14]] * 3
    bias.data = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        moe.moe_nvfp4_route_scored(lg, router, 2)
