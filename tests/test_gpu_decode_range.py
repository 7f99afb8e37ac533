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


def check_terms(ly, o, b, h, scale, what=""):
    """O of one head against 64 bits, to an error in proportion to sum p |v| and not to the largest |v|: each term is off
    by half a step of its weight's type (2^-11 for 8-bit pools, 2^-16 for bf16 ones) and by its logit's error, the sums by
    a rounding a term, O by half a step of bf16. Weights of 8-bit pools have a smallest step: they
    are off by up to 2^-25 units, of which the head's largest p 2^(y - 127) is 2^3 at least, times a code of M at most: by
    2^-27 of the largest p max|v|, since a row's largest code is above M / 2 (a little less where it was rounded)."""
    kv, vis = h // (ly.hq // ly.hkv), visible(ly, b, h)
    s, d = logits(ly, ly.stored(ly.k), b, h, scale)
    v = ly.stored(ly.v)[vis, kv].astype(np.float64)
    p = np.exp(s - s.max())
    p /= p.sum()
    want, total, n = p @ v, p @ np.abs(v), len(vis)
    rel = (2.0 ** -16 if ly.fmt == "bf16" else 2.0 ** -11) + 4 * (d + 2.0 ** -22 + np.abs(s).max() * 2.0 ** -23) + 2 * n * 2.0 ** -24
    floor = 0 if ly.fmt == "bf16" else 1.02 * n * 2.0 ** -27 * (p * np.abs(v).max(1)).max()
    tol = np.abs(want) * 2.0 ** -8 * (1 + 2.0 ** -8) + total * rel + floor
    err = np.abs(o[b, h] - want)
    assert (err <= tol).all(), f"{what} b={b} h={h}: off by {(err / tol).max():.1f} tolerances, {(err / total).max():.2e} of sum p|v|"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("down,up", [(60, 30), (90, 60), (20, 25), (110, 100)])
def test_a_huge_value_of_little_weight_leaves_the_others_theirs(down, up, fmt):
    """One visible value 2^up times the others at a logit `down` log2 units below them: O is still the others'."""
    ly = Layer([(1500, 1), (700, 3), (129, 1)], 8, 2, 128, 32, [[GLOBAL, local(140, 200)]] * 3, fmt, seed=400 + up)
    base = bf16(ly.rng.choice([-1.0, 1.0], (2, ly.D)))
    ly.q = bf16(np.repeat(base, 4, 0)[None] * ly.rng.choice([1.0, 1.25, 1.5], (3, 8, 1)))
    ly.k = bf16(ly.rng.standard_normal(ly.k.shape) * 0.25)
    scale = down / math.log2(math.e) / ly.D
    for b, at in enumerate((0, 650, 128)):
        ly.k[ly.cu[b] + at] = -base
        ly.v[ly.cu[b] + at] = bf16(ly.v[ly.cu[b] + at] * np.float32(2.0 ** up))
    o, _ = run(ly, scale)
    for b in range(ly.B):
        for h in range(ly.hq):
            check_terms(ly, o, b, h, scale, f"{fmt} {down} {up}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("D,P,lengths,G", [(128, 64, (3000, 40, 1), 4), (64, 16, (900, 257, 33), 4), (128, 128, (20001,), 4),
                                           (128, 32, (2500, 333), 16), (64, 64, (2000,), 32), (64, 16, (200,), 8),
                                           (128, 128, (250,), 1)])
def test_weights_and_values_that_make_up_for_one_another(D, P, lengths, G, order, fmt):
    """Logits over 100 log2 units, and values over 2^-100 the other way: every key counts about the same in one head, in
    others the largest logits or the largest values win."""
    ly = Layer([(n, 1) for n in lengths], 2 * G, 2, D, P, [[GLOBAL, local(150, 300)]] * len(lengths), fmt, seed=500)
    base = bf16(ly.rng.choice([-1.0, 1.0], (2, D)))
    slopes = np.resize([1.0, 0.5, 0.75, 1.0, 0.25, 0.9375, 0.0], 2 * G)
    ly.q = bf16(np.repeat(base, G, 0)[None] * slopes[None, :, None] * np.ones((ly.B, 1, 1)))
    ramp = np.concatenate([np.linspace(0, 1, n) if n > 1 else np.ones(1) for n in lengths])
    if order == "down":
        ramp = 1 - ramp
    elif order == "mixed":
        ramp = np.concatenate([ly.rng.permutation(x) for x in np.split(ramp, ly.cu[1:-1])])
    ly.k = bf16(ramp[:, None, None] * base[None])
    scale = 100 / math.log2(math.e) / D
    stored = ly.stored(ly.k)[:, 0, 0] * base[0, 0]                        # the ramp as the pool holds it
    ly.v = bf16(ly.v * np.exp2(50 - np.round(100 * stored)).astype(np.float32)[:, None, None])
    o, _ = run(ly, scale)
    for b in range(ly.B):
        for h in range(ly.hq):
            check_terms(ly, o, b, h, scale, f"{fmt} {order}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("share", [0.02, 0.5, 1.0])
def test_value_rows_of_zeros(share, fmt):
    """Rows of zeros, the most probable key's among them, beside ordinary and very small ones; and nothing but zeros."""
    ly = Layer([(1100, 1), (90, 1)], 8, 2, 128, 64, [[GLOBAL, local(100, 150)]] * 2, fmt, seed=600)
    zero = ly.rng.random(ly.v.shape[:2]) < share
    for b in range(2):
        for h in range(8):
            s, _ = logits(ly, ly.stored(ly.k), b, h, 0.3)
            zero[visible(ly, b, h)[int(np.argmax(s))], h // 4] = True
    ly.v[zero] = 0
    ly.v[5::7] = bf16(ly.v[5::7] * np.float32(2.0 ** -40))
    o, _ = run(ly, 0.3)
    for b in range(2):
        for h in range(8):
            check_terms(ly, o, b, h, 0.3, f"{fmt} {share}")


@pytest.mark.parametrize("fmt", FMTS)
def test_a_visible_nan_beside_values_of_very_different_size(fmt):
    """NaN reaches the heads that see it, and no others, where the values of a chunk span most of the float range."""
    ly = Layer([(700, 1), (300, 1)], 8, 2, 64, 32, [[GLOBAL, GLOBAL]] * 2, fmt, seed=601)
    ly.v = bf16(ly.v * np.exp2(ly.rng.uniform(-60, 20, ly.v.shape[:2] + (1,))).astype(np.float32))
    clean = Layer([(700, 1), (300, 1)], 8, 2, 64, 32, [[GLOBAL, GLOBAL]] * 2, fmt, seed=601)
    clean.v = ly.v.copy()
    ly.k[100, 1, 3] = np.nan                 # sequence 0, KV head 1: query heads 4..7
    ly.v[700 + 7, 0, 9] = np.inf             # sequence 1, KV head 0: query heads 0..3
    t = ly.upload(poison=False)
    o, lse = (x.float().cpu().numpy().astype(np.float64) for x in ly.decode(t, scale=0.1))
    assert np.isnan(o[0, 4:]).all() and np.isnan(lse[4:, 0]).all() and np.isfinite(lse[:, 1]).all()
    assert (~np.isfinite(o[1, :4, 9])).all()
    for b, hs in ((0, range(4)), (1, range(4, 8))):
        for h in hs:
            check_terms(clean, o, b, h, 0.1, fmt)
