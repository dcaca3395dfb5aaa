"""Pins of the oracle's MXFP4 quantisation and of its routing by scores: hand values, brute
force, torch, and finite differences."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from workloads import gen


# ----------------------------------------------------------------------------- MXFP4

def test_round_e2m1_grid_and_ties():
    v = np.array([0.0, 0.25, 0.26, 0.75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 6.0, 7.9, -0.75, -5.0])
    want = np.array([0.0, 0.0, 0.5, 1.0, 1.0, 1.5, 2.0, 2.0, 3.0, 4.0, 4.0, 6.0, 6.0, 6.0, -1.0, -4.0])
    assert np.array_equal(O.decode_e2m1(O.round_e2m1(v)), want)


@pytest.mark.parametrize("amax,byte", [(0.0, 0), (1.0, 125), (1.999, 125), (2.0, 126), (6.0, 127), (8.0, 128),
                                       (2.0 ** -126, 0), (2.0 ** -140, 0), (2.0 ** -124, 1), (2.0 ** 127, 252),
                                       (3.4e38, 252), (np.inf, 255), (np.nan, 255)])
def test_mxfp4_scale_byte(amax, byte):
    assert O.mxfp4_scale_byte(np.array([amax]))[0] == byte


def test_quantize_mxfp4_matches_the_workload_generator():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(7, 96, generator=g) * torch.exp2(torch.randint(-20, 20, (7, 1), generator=g).float())
    x[2, 32:64] = 0
    q, sf = O.quantize_mxfp4(x.numpy())
    pq, psf = gen._to_mxfp4(x.t().contiguous())              # [N, K/2], [K/32, N]
    assert np.array_equal(q, pq.numpy()) and np.array_equal(sf, psf.numpy().T)


def test_quantize_mxfp4_bad_blocks_and_layout():
    x = np.zeros((1, 96))
    x[0, 0], x[0, 1] = 1.0, -6.0                             # scale 1: codes 2 and 15
    x[0, 40] = np.nan
    x[0, 70] = -np.inf
    q, sf = O.quantize_mxfp4(x)
    assert list(sf[0]) == [127, 255, 255]
    assert q[0, 0] == (2 | (15 << 4)) and not q[0, 1:].any()
    assert np.isnan(O.decode_mxfp4_rows(q, sf)[0, 32:]).all()


# ----------------------------------------------------------------------------- routing by scores

def test_route_scored_without_extras_is_route_topk():
    lg = np.random.default_rng(0).standard_normal((20, 13)).astype(np.float32)
    idx, w = O.route_scored(lg, 4, score="softmax")
    ri, rw = O.route_topk(lg, 4)
    assert np.array_equal(idx, ri) and np.allclose(w, rw, atol=1e-15)


def test_route_scored_hand_example():
    # two groups of three; logit(0.5) = 0
    lg = np.log(np.array([[0.9, 0.2, 0.1, 0.6, 0.55, 0.5]]) / (1 - np.array([[0.9, 0.2, 0.1, 0.6, 0.55, 0.5]])))
    kw = dict(score="sigmoid", groups=2, topk_groups=1)
    idx, w = O.route_scored(lg, 2, group_top=1, **kw)         # group maxima .9 and .6
    assert list(idx[0]) == [0, 1] and np.allclose(w[0], [0.9 / 1.1, 0.2 / 1.1])
    idx, w = O.route_scored(lg, 2, group_top=2, **kw)         # sums 1.1 and 1.15
    assert list(idx[0]) == [3, 4]
    b = np.array([0, 0.5, 0, 0, 0, 0])                        # sums 1.6 and 1.15; choices .9, .7
    idx, w = O.route_scored(lg, 2, group_top=2, bias=b, renorm=False, scale=2.0, **kw)
    assert list(idx[0]) == [0, 1] and np.allclose(w[0], [1.8, 0.4])   # weights without the bias


def test_route_scored_masks():
    lg = np.array([[1.0, np.nan, -np.inf, np.finfo(np.float32).min, 0.5], [-np.inf] * 5])
    for score in ("softmax", "sigmoid"):
        idx, w = O.route_scored(lg, 3, score=score)
        assert idx.tolist() == [[0, 4, -1], [-1, -1, -1]]
        assert w[0, 2] == 0 and abs(w[0].sum() - 1) < 1e-12 and not w[1].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_scored_backward_matches_finite_differences(score, renorm):
    rng = np.random.default_rng(5)
    lg = rng.standard_normal((3, 6))
    lg[1, 2] = -np.inf
    kw = dict(score=score, renorm=renorm, scale=1.7)
    idx, _ = O.route_scored(lg, 3, **kw)
    d = rng.standard_normal((3, 3))
    got = O.route_scored_backward(lg, idx, d, **kw)

    def loss(x):
        s = O.scores(O.masked_logits(x, np.finfo(np.float32).min), score)
        p = np.take_along_axis(s, idx.astype(int), axis=1)
        if renorm:
            p = p / p.sum(axis=1, keepdims=True)
        return 1.7 * (p * d).sum()

    h = 1e-6
    for t in range(3):
        for e in range(6):
            if np.isinf(lg[t, e]):
                assert got[t, e] == 0
                continue
            a, b = lg.copy(), lg.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((loss(a) - loss(b)) / (2 * h) - got[t, e]) < 1e-8


def test_route_scored_backward_same_expert_twice_and_bad_ids():
    lg = np.array([[0.3, -0.2, 0.9]])
    kw = dict(score="sigmoid", renorm=False)
    one = O.route_scored_backward(lg, np.array([[2, -1]]), np.array([[3.0, 99.0]]), **kw)
    two = O.route_scored_backward(lg, np.array([[2, 2]]), np.array([[1.0, 2.0]]), **kw)
    assert np.allclose(one, two) and one[0, 0] == 0
