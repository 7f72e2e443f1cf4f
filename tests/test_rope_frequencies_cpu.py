"""rope_frequencies against separately written definitions of its scalings (CPU)."""
import math

import pytest
import torch

from speculative_decoding_05_b200.kv import rope_frequencies


def turns(i, rot, theta, original_len):
    """How often pair i turns over original_len positions, unscaled."""
    return original_len * theta ** (-2.0 * i / rot) / (2 * math.pi)


def near(got, want):
    """fp64 on both sides: a power and a handful of operations."""
    return all(abs(g - w) <= 1e-12 * abs(w) for g, w in zip(got.tolist(), want)) \
        and len(got) == len(want) and got.dtype == torch.float64


def yarn_plain(rot, theta, factor, original_len, fast, slow):
    """The published interpolation, pair by pair: the index at which a pair turns
    r times is rot ln(len / (2 pi r)) / (2 ln theta); the lower bound is that of
    `fast` turns rounded down, at least 0, the upper that of `slow` turns rounded
    up, at most rot - 1; frequencies are kept below the one, divided by factor
    above the other, mixed in between."""
    def at(r):
        return rot * math.log(original_len / (2 * math.pi * r)) / (2 * math.log(theta))

    a, b = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
    out = []
    for i in range(rot // 2):
        f = 1.0 / theta ** (2.0 * i / rot)
        t = min(max((i - a) / (b - a), 0.0), 1.0)
        out.append((1.0 - t) * f + t * f / factor)
    return out


@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("theta", [1e4, 5e5, 1e6])
def test_plain_and_linear(rot, theta):
    want = [math.exp(-2.0 * i / rot * math.log(theta)) for i in range(rot // 2)]
    f, scale = rope_frequencies(rot, theta)
    assert near(f, want) and scale == 1.0
    f, scale = rope_frequencies(rot, theta, "linear", 8.0)
    assert near(f, [w / 8.0 for w in want]) and scale == 1.0


@pytest.mark.parametrize("rot", [2, 16, 64, 128])
@pytest.mark.parametrize("factor", [1.0, 2.0, 8.0])
def test_ntk_keeps_the_highest_and_divides_the_lowest(rot, factor):
    theta = 1e4
    f, scale = rope_frequencies(rot, theta, "ntk", factor)
    assert scale == 1.0 and f[0] == 1.0
    if rot > 2:
        last = theta ** (-(rot - 2.0) / rot) / factor
        ratio = last ** (1.0 / (rot // 2 - 1))  # a geometric row from 1 to that
        assert near(f, [ratio ** i for i in range(rot // 2)])


@pytest.mark.parametrize("rot,theta,original_len", [
    (128, 1e4, 4096), (128, 1e6, 32768), (64, 1e4, 256), (64, 5e5, 8192),
    # the last pair turns more than beta_slow times: the ramp ends beyond it
    (128, 1e4, 65536), (128, 1e4, 131072), (64, 1e4, 131072), (32, 1e4, 262144),
])
@pytest.mark.parametrize("factor", [2.0, 4.0, 40.0])
def test_yarn(rot, theta, original_len, factor):
    f, scale = rope_frequencies(rot, theta, "yarn", factor, original_len)
    assert near(f, yarn_plain(rot, theta, factor, original_len, 32.0, 1.0))
    assert abs(scale - (0.1 * math.log(factor) + 1.0)) < 1e-15
    f, _ = rope_frequencies(rot, theta, "yarn", factor, original_len, 16.0, 2.0)
    assert near(f, yarn_plain(rot, theta, factor, original_len, 16.0, 2.0))


def test_yarn_divides_no_pair_by_the_whole_factor_that_turns_often_enough():
    """A pair that turns more than beta_slow times lies between the bounds."""
    rot, theta, n = 128, 1e4, 131072
    f, _ = rope_frequencies(rot, theta, "yarn", 4.0, n)
    last = rot // 2 - 1
    assert turns(last, rot, theta, n) > 2.0
    ratio = float(f[last]) / theta ** (-2.0 * last / rot)
    assert 0.4 < ratio < 0.5  # 0.46; 0.25 is the whole factor
    fast = [i for i in range(rot // 2) if turns(i, rot, theta, n) > 32.0]
    assert fast and all(abs(float(f[i]) * theta ** (2.0 * i / rot) - 1.0) < 1e-12 for i in fast[:-1])


@pytest.mark.parametrize("factor", [0.25, 0.5, 1.0])
def test_yarn_without_stretching_keeps_the_attention_factor(factor):
    """The published attention factor is 1 unless positions are stretched."""
    assert rope_frequencies(64, 1e4, "yarn", factor, 4096)[1] == 1.0


@pytest.mark.parametrize("bad", [dict(rot_dim=0), dict(rot_dim=15), dict(rot_dim=-4),
                                 dict(rot_dim=64, scaling="cubic"),
                                 dict(rot_dim=64, scaling="yarn", factor=4.0)])
def test_refusals(bad):
    with pytest.raises(ValueError):
        rope_frequencies(**bad)
