"""The error bounds that moe_route_scored's fp32 routing rests on, checked by arithmetic against the constants in the
kernel's source: the difference of two fp32 scores (or sums of two) is off by less than what the kernels allow for, in
the worst case that the roundings permit.

All in units u = 2^-23.  exp(x) is off by at most (0.61 |x| + 1) u of its value: the product with log2(e) and that constant's
own rounding move the exponent by 0.61 |x| u, the instruction is good to one ulp.  Rounding l - max adds 0.5 |x|."""
import math
import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0**-23


def source():
    return open(os.path.join(ROOT, "bit_moe_expert_top_amd", "csrc", "block", "route_scored.hip")).read()


def power(text):
    return 1.0 / float(eval(re.fullmatch(r"1\.0f / \((1 << \d+)\)", text).group(1)))


def near(vpl):
    m = re.search(r"kNear = VPL > 8 \? (1\.0f / \(1 << \d+\)) : (1\.0f / \(1 << \d+\));", source())
    return power(m.group(1 if vpl > 8 else 2))


def exact(sigmoid):
    m = re.search(r"kExact = SIGMOID \? (1\.0f / \(1 << \d+\)) : (1\.0f / \(1 << \d+\))", source())
    return power(m.group(1 if sigmoid else 2))


def own(m, x, p):
    """A candidate's own bound in route_rows_kernel, softmax, x = max - l."""
    c = re.search(r"p \* \((?:([0-9.]+)f \* \()?lmax - le\)? \+ (?:\(?(\d+) \* M \+ (\d+)\)?|([0-9.]+)f)\)", source())
    slope = float(c.group(1) or 1)
    const = float(c.group(4)) if c.group(4) else int(c.group(2)) * m + int(c.group(3))
    return p * (slope * x + const) * U


def common(terms, lanes_steps, experts):
    """The error of the softmax's 1 / sum, the same for every score of a token: the additions, the terms' own errors, each
    weighted by its p (sum of p |x| = entropy - log(sum) <= ln E), the reciprocal."""
    return (0.5 * (terms - 1 + lanes_steps) + 1.11 * math.log(experts) + 1 + 0.5) * U


def score_error(x, p):
    """What is a softmax score's own: its exponential's error and the product's rounding."""
    return p * (1.11 * x + 1 + 0.5) * U


def pairs(seed, n=200000):
    """Two scores of a token: x = max - l of both and their p, exp(-x) / sum with a sum of at least both."""
    r = np.random.default_rng(seed)
    xa, xb = (np.where(r.random(n) < 0.2, 0.0, r.exponential(r.choice([0.1, 1, 10], size=n))) for _ in range(2))
    rest = r.exponential(r.choice([1e-6, 0.1, 1, 100], size=n))
    z = np.maximum(np.exp(-xa) + np.exp(-xb) + rest, 1.0)
    return xa, xb, np.exp(-xa) / z, np.exp(-xb) / z


@pytest.mark.parametrize("m", [1, 2, 3, 4])
def test_candidates_own_bounds(m):
    xa, xb, pa, pb = pairs(m)
    worst = score_error(xa, pa) + score_error(xb, pb) + common(8 * m, 4, 128 * m) * np.abs(pa - pb)
    assert (worst <= own(m, xa, pa) + own(m, xb, pb)).all()


@pytest.mark.parametrize("m", [1, 2, 3, 4])
def test_rows_kernel_bound(m):
    """Sums of two scores in each of two groups: four scores that sum to 1 at most, p x summing to 0.72 at most."""
    assert common(8 * m, 4, 128 * m) + (1.5 + 1.11 * 0.72) * U <= exact(False)
    sigmoid = 4 * (0.25 * 1 + 0.61 * 0.224 + 1.5) * U  # p (1 - p) (0.61 |l| + 1) + 1.5 p
    assert sigmoid <= exact(True)


@pytest.mark.parametrize("vpl,bits", [(1, 0), (2, 1), (4, 2), (6, 3), (8, 3), (16, 4)])
def test_token_kernel_bound(vpl, bits):
    score = common(vpl, 6, 64 * vpl) + (1.5 + 1.11 * 0.72) * U
    assert score <= near(vpl) and 4 * (0.25 + 0.61 * 0.224 + 1.5) * U <= near(vpl)
    # adding the biases, half an ulp of each c, and dropping bits of the lower one
    assert (1 + 2**bits) * U <= near(vpl)


def test_four_scores_times_their_distance():
    """p x of four experts sums to at most 0.72: it is largest for equal x, where 4 x e^-x / (1 + 4 e^-x) has its maximum
    W(4 / e) = 0.7177 (at x = 1 + W(4 / e), W being Lambert's function)."""
    assert abs(0.7177 * math.exp(0.7177) - 4 / math.e) < 1e-3
    r = np.random.default_rng(3)
    x = r.exponential(2.0, size=(200000, 4))
    p = np.exp(-x) / (1 + np.exp(-x).sum(1, keepdims=True))
    assert (x * p).sum(1).max() <= 0.72
    x[:, 0] = 0  # one of them the largest
    p = np.exp(-x) / np.exp(-x).sum(1, keepdims=True)
    assert (x * p).sum(1).max() <= 0.72
