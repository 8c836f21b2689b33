"""Pins of the oracle of the operators around the expert FFN: hand-worked values, torch's own
functions, brute force."""
import math

import numpy as np
import torch

from oracle import block as OB
from oracle import moe as OM


def test_norm_by_hand():
    x = np.array([[3.0, 4.0, 0.0, 0.0]], np.float32)
    s, y = OB.add_rmsnorm(x, None, np.array([1.0, 2.0, 1.0, 1.0]), 1e-30, False)
    assert np.array_equal(s, x)
    np.testing.assert_allclose(y, [[3 / 2.5, 2 * 4 / 2.5, 0, 0]], rtol=1e-15)
    # the norm is taken of the rounded sum: 256 + 1 is a tie between the bf16 values 256 and 258
    s, y = OB.add_rmsnorm([[256.0, 0.0]], [[1.0, 0.0]], np.ones(2), 1e-30, True)
    assert s.tolist() == [[256.0, 0.0]]
    s, _ = OB.add_rmsnorm([[256.0, 0.0]], [[1.0, 0.0]], np.ones(2), 1e-30, False)
    assert s.tolist() == [[257.0, 0.0]]


def test_bf16_round_against_torch():
    v = np.random.default_rng(0).normal(size=4096).astype(np.float32) * 1e3
    assert np.array_equal(OB.bf16_round(v), torch.from_numpy(v).bfloat16().float().numpy())


def test_norm_of_unit_weight_has_unit_rms():
    x = np.random.default_rng(1).normal(size=(5, 96)).astype(np.float32)
    _, y = OB.add_rmsnorm(x, None, np.ones(96), 1e-30, False)
    np.testing.assert_allclose((y * y).mean(axis=1), 1.0, rtol=1e-12)


def test_activations_against_torch():
    a = np.linspace(-30, 30, 241)[None]
    t = torch.from_numpy(a)
    for name, f in (("relu", torch.relu), ("silu", torch.nn.functional.silu),
                    ("gelu", lambda v: torch.nn.functional.gelu(v, approximate="tanh"))):
        # torch's gelu forms 1 + tanh u, which near u = -inf is off by a few 2^-53: |a| <= 30 times that
        np.testing.assert_allclose(OB.act(a, name), f(t).numpy(), rtol=1e-12, atol=30 * 3 * 2.0**-53)
    two = np.concatenate([a, a[:, ::-1]], axis=1)
    np.testing.assert_allclose(OB.act(two, "swiglu"), OB.act(a, "silu") * a[:, ::-1], rtol=1e-14)


def test_linear_by_hand():
    out = OB.linear([[1.0, 2.0]], [[3.0, 4.0], [-5.0, 1.0]], bias=[0.5, 0.0], act_name="relu", residual=[[1.0, 7.0]])
    assert out.tolist() == [[12.5, 7.0]]


def test_scored_routing_by_hand():
    lg = np.log(np.array([[1.0, 2.0, 3.0, 4.0]], np.float32))  # softmax: .1 .2 .3 .4
    ids, g = OB.route_scored(lg, 2, "softmax", scale=2.0)
    assert ids.tolist() == [[3, 2]]
    np.testing.assert_allclose(g, [[0.8, 0.6]], rtol=1e-6)
    # the bias moves the choice and not the gates
    ids, g = OB.route_scored(lg, 2, "softmax", bias=[0.35, 0, 0, 0], renormalize=True)
    assert ids.tolist() == [[0, 3]]
    np.testing.assert_allclose(g, [[0.2, 0.8]], rtol=1e-6)
    # groups (0,1) and (2,3): by their best the second, by their two best with this bias the first
    bias = [0.1, 0.3, 0.0, 0.05]  # c = .2 .5 .3 .45
    assert OB.route_scored(lg, 1, "softmax", bias=bias, n_group=2)[0].tolist() == [[1]]
    assert OB.route_scored(lg, 2, "softmax", bias=bias, n_group=2, group_top=2)[0].tolist() == [[3, 2]]
    # out of service: last, with gate 0
    ids, g = OB.route_scored(lg, 4, "softmax", bias=[0, 0, 0, -np.inf], renormalize=True)
    assert ids.tolist() == [[2, 1, 0, 3]] and g[0, 3] == 0.0
    np.testing.assert_allclose(g[0, :3], [0.5, 1 / 3, 1 / 6], rtol=1e-6)
    # nothing left: the lowest ids, gates 0
    ids, g = OB.route_scored(np.full((1, 4), -np.inf, np.float32), 2, "softmax", renormalize=True)
    assert ids.tolist() == [[0, 1]] and g.tolist() == [[0.0, 0.0]]


def test_renormalised_softmax_without_bias_is_the_plain_routing():
    lg = np.random.default_rng(3).normal(size=(40, 24)).astype(np.float32)
    lg[::3] = np.round(lg[::3])  # ties
    ids, g = OB.route_scored(lg, 5, "softmax", renormalize=True)
    want, gw = OM.route(lg, 5)
    assert np.array_equal(ids, want)
    np.testing.assert_allclose(g, gw, rtol=1e-12)


def test_groups_against_a_search_over_all_sets():
    import itertools

    r = np.random.default_rng(4)
    lg, bias = r.normal(size=(20, 12)).astype(np.float32), r.normal(size=12).astype(np.float32) * 0.2
    c = OB.scores(lg, "sigmoid") + bias.astype(np.float64)
    for top in (1, 2):
        ids, _ = OB.route_scored(lg, 4, "sigmoid", bias=bias, n_group=4, topk_group=2, group_top=top)
        for t in range(20):
            value = [sum(sorted(c[t, 3 * g:3 * g + 3])[-top:]) for g in range(4)]
            best = max(itertools.combinations(range(4), 2), key=lambda s: sum(value[g] for g in s))
            pool = [e for e in range(12) if e // 3 in best]
            assert sorted(ids[t]) == sorted(sorted(pool, key=lambda e: -c[t, e])[:4])
    assert math.isclose(float(c[0, 0]), 1 / (1 + math.exp(-float(lg[0, 0]))) + float(bias[0]), rel_tol=1e-12)
