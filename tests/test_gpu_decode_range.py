"""Single-token attention where the plain formula is easy to get wrong in 32 bits: logits far from 0, whose product with
the scale rounds by more than a unit, and softmaxes whose weights or values span most of the float range."""
import math

import numpy as np
import pytest
import torch

from decode_common import GLOBAL, Layer, bf16, check_attention, local
from oracle import reference as orc

pytestmark = pytest.mark.gpu
FMTS = ("bf16", "e4m3", "int8")


def run(ly, scale):
    t = ly.upload()
    o, lse = ly.decode(t, scale=scale)
    assert int(t["status"].item()) == 0
    return o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def visible(ly, b, h):
    """Row numbers (in ly.k) of the keys that sequence b's last position sees through query head h."""
    c = ly.cls[b, h // (ly.hq // ly.hkv)]
    return int(ly.cu[b]) + orc.visible_keys(*(int(x) for x in c), int(ly.L[b]) - 1)


def logits(ly, k, b, h, scale):
    """(logits of those keys, bound on their error in fp32: sums of D products, then a few roundings) in 64 bits. k: the
    keys as they are stored."""
    k = k[visible(ly, b, h), h // (ly.hq // ly.hkv)].astype(np.float64)
    q = ly.q[b, h].astype(np.float64)
    return k @ q * scale, (ly.D + 8) * 2.0 ** -24 * float((np.abs(k) @ np.abs(q)).max()) * abs(scale)


def check_lse(lse, want, d):
    # the logit's own error, and a few roundings of the result (each half of 2^-23 of it)
    assert abs(lse - want) <= d + abs(want) * 2.0 ** -21 + 2.0 ** -20, (lse, want, d)


SIZES = [10, 20, 24, 26, 29, 34, 60]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", SIZES)
def test_one_visible_key_returns_its_value(size, fmt):
    """A softmax over one key is 1 whatever the logit: O is that key's value, which bf16 holds exactly."""
    classes = [[GLOBAL, local(0, 1)]] * 12 + [[local(0, 1), local(0, 1)]] * 20
    ly = Layer([(1, 1)] * 12 + [(100 + 7 * i, 1) for i in range(20)], 16, 2, 128, 32, classes, fmt, seed=size)
    scale = 2.0 ** size / math.sqrt(ly.D)
    o, lse = run(ly, scale)
    k, v = ly.stored(ly.k), ly.stored(ly.v)
    for b in range(ly.B):
        for h in range(ly.hq):
            s, d = logits(ly, k, b, h, scale)
            assert len(s) == 1
            np.testing.assert_array_equal(o[b, h], v[ly.cu[b + 1] - 1, h // 8])
            check_lse(lse[h, b], s[0], d)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,G", [(128, 8), (64, 4), (128, 16)])
@pytest.mark.parametrize("size", SIZES)
def test_equal_keys_weigh_the_same(size, D, G, fmt):
    """All keys equal: every logit is the same number, and O is the mean of the visible values, over one tile as over many
    tiles in many blocks."""
    ly = Layer([(5, 1), (131, 1), (3077, 1)], 2 * G, 2, D, 64, [[GLOBAL, local(130, 200)]] * 3, fmt, seed=100 + size)
    for b in range(ly.B):
        ly.k[ly.cu[b]:ly.cu[b + 1]] = ly.k[ly.cu[b]]
    scale = 2.0 ** size / math.sqrt(D)
    o, lse = run(ly, scale)
    k, v = ly.stored(ly.k), ly.stored(ly.v).astype(np.float64)
    for b in range(ly.B):
        for h in range(ly.hq):
            s, d = logits(ly, k, b, h, scale)
            vis = v[visible(ly, b, h), h // G]
            want, n = vis.mean(0), len(vis)
            # O is rounded to bf16; the weights are equal and exact, the sums of n terms are off by n roundings at most
            tol = np.abs(want) * (2.0 ** -8 + 2.0 ** -16) + np.abs(vis).mean(0) * 2 * n * 2.0 ** -24
            assert (np.abs(o[b, h] - want) <= tol).all(), (b, h, np.abs(o[b, h] - want).max())
            check_lse(lse[h, b], s[0] + math.log(n), d)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("hot", [0, 130, -1])
def test_one_hot_at_any_size(hot, size, fmt):
    """One key far above the others: O is its value exactly, however large the logit."""
    ly = Layer([(2500, 1), (2500, 2)], 8, 2, 64, 16, [[GLOBAL, local(140, 150)]] * 2, fmt, seed=200 + size)
    base = bf16(ly.rng.choice([-1.0, 1.0], (2, ly.D)))             # per KV head; q and k are multiples of it
    ly.q = bf16(np.repeat(base, 4, 0)[None] * ly.rng.choice([1.0, 1.25, 1.5], (2, 8, 1)))
    ly.k = bf16(base[None] * ly.rng.choice([-1.0, 0.25, 0.5, 1.0], (5000, 2, 1)))
    hot %= 2500
    ly.k[[hot, 2500 + hot]] = bf16(1.75 * base)
    scale = 2.0 ** size / ly.D                                     # logits 1.75 c 2^size against c 2^size at most
    o, lse = run(ly, scale)
    k, v = ly.stored(ly.k), ly.stored(ly.v)
    for b in range(2):
        for h in range(8):
            s, d = logits(ly, k, b, h, scale)
            np.testing.assert_array_equal(o[b, h], v[2500 * b + hot, h // 4])
            check_lse(lse[h, b], s.max(), d)


@pytest.mark.parametrize("fmt", FMTS)
def test_a_scale_of_zero_ignores_the_keys(fmt):
    """0 q.k = 0 for any finite keys: O is the mean of the values, also where q.k is near the end of the float range."""
    ly = Layer([(300, 1), (77, 1)], 8, 2, 64, 16, [[GLOBAL, local(20, 30)]] * 2, fmt, seed=301)
    ly.q = bf16(ly.q * np.float32(2.0 ** 60))
    ly.k = bf16(ly.k * np.float32(2.0 ** 55))
    v = ly.stored(ly.v).astype(np.float64)
    for scale in (0.0, 1e-45):
        o, lse = run(ly, scale)
        for b in range(2):
            for h in range(8):
                vis = v[visible(ly, b, h), h // 4]
                want, n = vis.mean(0), len(vis)
                tol = np.abs(want) * (2.0 ** -8 + 2.0 ** -16) + np.abs(vis).mean(0) * (2 * n * 2.0 ** -24 + 2.0 ** -16)
                assert (np.abs(o[b, h] - want) <= tol).all(), (scale, b, h)
                check_lse(lse[h, b], math.log(n), 2.0 ** -20)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("k_scale,scale", [(2.0 ** 118, 2.0 ** -120), (2.0 ** 100, -2.0 ** -102), (2.0 ** -118, 2.0 ** 106)])
def test_keys_near_the_ends_of_the_float_range(k_scale, scale, fmt):
    """Keys that only the scale brings to logits of ordinary size."""
    ly = Layer([(600, 1), (1, 1)], 8, 2, 128, 64, [[GLOBAL, local(20, 200)]] * 2, fmt, seed=302, k_scale=k_scale)
    t = ly.upload()
    check_attention(*ly.decode(t, scale=scale), ly.attention(scale), f"{fmt} {k_scale} {scale}")
