"""Routing where scores are not numbers or experts are missing, and the expert layer with more
routes than experts."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import q8_util as R  # noqa: E402
from test_gpu_route import DEV, DT, Layer, check  # noqa: E402

tern = pytest.importorskip("ternary_weight_matmul_amd")

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,keep,best", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("renorm", [False, True])
def test_logits_that_are_not_finite(score, biased, groups, keep, best, renorm):
    """A softmax over +inf or NaN has NaN weights, whichever experts are taken."""
    E = 32
    rng = np.random.default_rng(11)
    lg = torch.from_numpy(rng.standard_normal((6, E))).float()
    lg[0, 3] = INF
    lg[1, 29], lg[1, 30] = INF, INF
    lg[2, 17] = NAN
    lg[3, 8:] = -INF
    lg[3, 5] = INF
    lg[4, :31], lg[4, 31] = -INF, NAN
    bias = torch.from_numpy(rng.standard_normal(E) * 0.1).float() if biased else None
    check(lg, 8, score, bias, groups, keep, best, renorm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("scale", [1.0, INF, -INF, NAN])
def test_places_without_an_expert_have_no_weight(score, biased, renorm, scale):
    """ids -1 come with weight 0, also beside NaN weights and with any factor."""
    E = 16
    lg = torch.full((4, E), -INF)
    lg[0, 2] = NAN
    lg[1, 4] = INF
    lg[2, 5], lg[2, 9] = 0.25, -1.5
    bias = torch.linspace(-0.1, 0.1, E) if biased else None
    ids, w = tern.moe_route(lg.to(DEV), 6, score=score, bias=bias.to(DEV) if biased else None, renormalize=renorm, scale=scale)
    want_ids, want = R.route(R.f64(lg), 6, score, R.f64(bias) if biased else None, 1, 1, 1, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = R.f64(w)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
    fine = np.isfinite(want)
    assert (np.abs(got[fine] - want[fine]) <= np.abs(want[fine]) * R.STEP * 1.001).all()
    assert (w[ids < 0] == 0).all()


@pytest.mark.parametrize("T,E,k", [(1, 3, 8), (4, 3, 8), (5, 3, 8), (70, 3, 8), (1, 1, 32), (4, 1, 32), (5, 1, 32), (70, 1, 32),
                                   (3, 5, 31), (20, 2, 17)])
@pytest.mark.parametrize("xd,yd", [("bf16", "bf16"), ("f16", "f32")])
def test_more_routes_than_experts(T, E, k, xd, yd):
    """An expert that is taken many times has the sum of its weights."""
    print(f"routed T={T} E={E} k={k} {xd}->{yd}", flush=True)
    H, F = 384, 256
    L = Layer(E, H, F, T + E)
    rng = np.random.default_rng(T + k)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(DT[xd])
    ids = torch.from_numpy(rng.integers(-1, E + 1, (T, k)).astype(np.int32))
    w = torch.from_numpy(rng.standard_normal((T, k))).float()
    want, bound = L.want(x, ids, w, yd)
    R.assert_close(L.run(x, ids, w, yd), want, bound, "more routes than experts")


def test_which_group_comes_first_where_scores_run_out_of_bits():
    """Sigmoids that are 1 in 64 bits: with one best expert and no bias groups go by logits, with two by scores."""
    lg = torch.tensor([[45.0, 44.0, 43.0, 42.0, 60.0, 41.0, 42.5, 50.0]]).to(DEV)
    ids, _ = tern.moe_route(lg, 2, score="sigmoid", groups=2, keep_groups=1, group_best=1)
    assert ids.tolist() == [[4, 7]]
    ids, _ = tern.moe_route(lg, 2, score="sigmoid", groups=2, keep_groups=1, group_best=2)
    assert ids.tolist() == [[0, 1]]


def test_a_group_with_one_open_expert_has_that_ones_score():
    lg = torch.tensor([[-INF, 3.0, -INF, -INF, 0.5, 0.25, 0.0, 0.75], [-INF, -1.0, -INF, -INF, 0.5, 0.25, 0.0, 0.75]]).to(DEV)
    for bias in (None, torch.zeros(8, device=DEV)):
        ids, w = tern.moe_route(lg, 3, score="sigmoid", bias=bias, groups=2, keep_groups=1, group_best=2)
        # 0.95 alone against 0.68 + 0.62, and 0.27 alone
        assert ids.tolist() == [[7, 4, 5], [7, 4, 5]]
    lg[0, 4:6], lg[0, 7] = -INF, -INF
    ids, w = tern.moe_route(lg, 3, score="sigmoid", groups=2, keep_groups=1, group_best=2)
    assert ids.tolist()[0] == [1, -1, -1] and w[0].tolist()[1:] == [0, 0]   # 0.95 against 0.5
