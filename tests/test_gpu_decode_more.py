"""Decode-side calls where a call that did nothing, or did it in the wrong place, would show: fresh rows on marked pools, codes
and exponent bytes in full; and layers with more pairs than threads, runs of many pairs, pages that heads share."""
import math

import numpy as np
import pytest
import torch

from decode_common import DTYPE, GLOBAL, Layer, bf16, check_attention, local
from head_sparse_paged_b200 import segpaged as sp
from oracle import reference as orc

pytestmark = pytest.mark.gpu
FMTS = ("bf16", "e4m3", "int8")


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def dev_bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(torch.bfloat16)


def raw(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype != torch.bfloat16 else t.float().cpu().numpy()


def same_codes(got, want, fmt):
    """Equal, but for the sign of an e4m3 zero, which is not part of its value."""
    if fmt == "e4m3":
        got, want = (np.where((x & 127) == 0, 0, x) for x in (got, want))
    np.testing.assert_array_equal(got, want)


def check_pools(ly, k, v, scale, want, where):
    """The pools' rows in the mask `where` [pages, P] against want, exponent bytes included."""
    for which, pool in enumerate((k, v)):
        same_codes(raw(pool)[where], want[which][0][where], ly.fmt)
        if ly.fmt != "bf16":
            np.testing.assert_array_equal(scale.cpu().numpy()[:, which][where], want[which][1][where])


def rows_at(ly, positions):
    """Mask [pages, P] of the stored rows of the given positions: a list for each sequence."""
    at = np.zeros((ly.num_pages, ly.P), bool)
    for b, ps in enumerate(positions):
        for h in range(ly.hkv):
            for p in ps:
                if p // ly.P in ly.pages[b][h]:
                    at[ly.table[ly.offs[b * ly.hkv + h] + ly.pages[b][h].index(p // ly.P)], p % ly.P] = True
    return at


@pytest.mark.parametrize("fmt", FMTS)
def test_append_of_fresh_rows_past_32_bits(fmt):
    """Rows that the pools did not hold, into pages beyond 2^31 elements: they land there, and nothing else changes."""
    ly = Layer([(700, 3), (129, 1)], 16, 2, 128, 128, [[GLOBAL, local(20, 200)]] * 2, fmt, seed=45)
    first = (1 << 31) // (ly.P * ly.D) + 3
    t = ly.upload(poison=False)
    dims = sp.Dims(ly.B, ly.hq, ly.hkv, ly.D, ly.P, first + ly.num_pages)

    def big(x):
        x = x.view(torch.uint8) if x.dtype != torch.bfloat16 else x
        out = torch.zeros((dims.num_pages, *x.shape[1:]), dtype=x.dtype, device="cuda")
        out[first:].copy_(x)
        return out

    k, v = (big(t[x]).view(t[x].dtype) for x in "kv")
    sc = None if fmt == "bf16" else big(t["scale"])
    k_new, v_new = (bf16(ly.rng.standard_normal((4, 2, 128)) * 3) for _ in range(2))
    sp.segpaged_append(dims, dev_bf16(k_new), dev_bf16(v_new), i32([0, 3, 4]), t["ctx"], t["lq"], t["cls"], t["table"] + first,
                       t["offs"], k, v, sc, t["status"])
    assert int(t["status"].item()) == 0
    ly.k[[697, 698, 699, 828]], ly.v[[697, 698, 699, 828]] = k_new, v_new
    want, used = ly.expected_pools()
    cut = [x.view(torch.uint8)[first:] if x.dtype != torch.bfloat16 else x[first:] for x in (k, v)]
    check_pools(ly, *cut, None if sc is None else sc[first:], want, np.broadcast_to(used[:, None], (ly.num_pages, ly.P)))
    for x in (k, v) + (() if sc is None else (sc,)):
        low = x.view(torch.uint8)[:first] if x.dtype != torch.bfloat16 else x[:first]
        assert not bool(low.any())


@pytest.mark.parametrize("fmt", FMTS[1:])
def test_build_past_32_bits_in_full(fmt):
    """K, V and exponent bytes of a build into marked pages beyond 2^31 elements, bit for bit."""
    ly = Layer([(700, 3), (129, 1)], 16, 2, 128, 128, [[GLOBAL, local(20, 200)]] * 2, fmt, seed=46)
    first = (1 << 31) // (ly.P * ly.D) + 3
    dims = sp.Dims(ly.B, ly.hq, ly.hkv, ly.D, ly.P, first + ly.num_pages)
    t = ly.upload(poison=False)
    k, v = (torch.full((dims.num_pages, ly.P, ly.D), 0x33, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.full((dims.num_pages, 2, ly.P), 0x33, dtype=torch.uint8, device="cuda")
    sp.segpaged_build_quant(dims, dev_bf16(ly.k), dev_bf16(ly.v), i32(ly.cu), t["lq"], t["cls"], t["table"] + first, t["offs"], None,
                            k.view(DTYPE[fmt]), v.view(DTYPE[fmt]), sc, t["status"])
    assert int(t["status"].item()) == 0
    want, used = ly.expected_pools()
    check_pools(ly, k[first:], v[first:], sc[first:], want, np.broadcast_to(used[:, None], (ly.num_pages, ly.P)))
    for x in (k, v, sc):
        assert bool((x[:first] == 0x33).all()) and bool((x[first:][torch.from_numpy(~used).cuda()] == 0x33).all())


@pytest.mark.parametrize("fmt", FMTS)
def test_append_of_fresh_rows_inside_a_larger_table(fmt):
    """Offsets that begin past 0 and end before the table does, rows that the pools did not hold."""
    ly = Layer([(300, 7), (65, 65)], 4, 2, 64, 32, [[GLOBAL, local(5, 40)], [local(0, 9), GLOBAL]], fmt, seed=47, spare=8)
    spare = np.setdiff1d(np.arange(ly.num_pages), ly.table)[:5]
    t = ly.upload(poison=False)
    before = [raw(t["k"]).copy(), raw(t["v"]).copy(), None if fmt == "bf16" else t["scale"].cpu().numpy().copy()]
    t["table"] = i32(np.concatenate([spare[:3], ly.table, spare[3:]]))
    t["offs"] += 3
    k_new, v_new = (bf16(ly.rng.standard_normal((5, 2, 64)) * 5) for _ in range(2))
    sp.segpaged_append(ly.dims(), dev_bf16(k_new), dev_bf16(v_new), i32([0, 3, 5]), t["ctx"], t["lq"], t["cls"], t["table"],
                       t["offs"], t["k"], t["v"], t["scale"], t["status"])
    assert int(t["status"].item()) == 0
    at = [297, 298, 299, 363, 364]
    ly.k[at], ly.v[at] = k_new, v_new
    new = rows_at(ly, [[297, 298, 299], [63, 64]])
    check_pools(ly, t["k"], t["v"], t["scale"], ly.expected_pools()[0], new)
    for got, old in zip((raw(t["k"]), raw(t["v"])), before):
        np.testing.assert_array_equal(got[~new], old[~new])
    if fmt != "bf16":
        np.testing.assert_array_equal(t["scale"].cpu().numpy().transpose(0, 2, 1)[~new], before[2].transpose(0, 2, 1)[~new])


@pytest.mark.parametrize("fmt", FMTS)
def test_append_drops_rows_and_writes_the_others_in_full(fmt):
    """More new rows than the window's pages hold: the kept ones with their exponent bytes, the others nowhere."""
    ly = Layer([(400, 1)], 2, 2, 64, 16, [[GLOBAL, local(10, 20)]], fmt, seed=48)
    t = ly.upload(poison=False)
    mark = 0x33 if fmt != "bf16" else 5.0
    for x in ("k", "v"):
        (t[x].view(torch.uint8) if fmt != "bf16" else t[x]).fill_(mark)
    if fmt != "bf16":
        t["scale"].fill_(mark)
    k_new, v_new = (bf16(ly.rng.standard_normal((400, 2, 64))) for _ in range(2))
    sp.segpaged_append(ly.dims(), dev_bf16(k_new), dev_bf16(v_new), i32([0, 400]), t["ctx"], t["lq"], t["cls"], t["table"],
                       t["offs"], t["k"], t["v"], t["scale"], t["status"])
    assert int(t["status"].item()) == 0
    ly.k, ly.v = k_new, v_new
    new = rows_at(ly, [list(range(400))])
    assert new.sum() == 400 + 16 + 32                       # the global head's, and the local head's three pages
    check_pools(ly, t["k"], t["v"], t["scale"], ly.expected_pools()[0], new)
    for x in (t["k"], t["v"]):
        assert (raw(x)[~new] == mark).all()
    if fmt != "bf16":
        assert (t["scale"].cpu().numpy().transpose(0, 2, 1)[~new] == mark).all()


def many(B, H):
    """B short sequences, some of them empty: lengths of 0 to 40."""
    return [(i * 7 % 41, min(1, i * 7 % 41)) for i in range(B)], [[GLOBAL] + [local(2, 3)] * (H - 1)] * B


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,H,G,D", [(150, 4, 1, 64), (300, 4, 2, 128), (1300, 4, 1, 64), (40, 2, 128, 64)])
def test_more_pairs_than_threads(B, H, G, D, fmt):
    """Several pairs a thread to count, runs of more pairs than a helper warp's window, and eight passes of one pair."""
    seqs, classes = many(B, H)
    ly = Layer(seqs, H * G, H, D, 16, classes, fmt, seed=49)
    t = ly.upload()
    o, lse = ly.decode(t)
    assert int(t["status"].item()) == 0
    check_attention(o, lse, ly.attention(1 / math.sqrt(D)), f"{fmt} {B} {H} {G} {D}")


@pytest.mark.parametrize("fmt", FMTS[1:])
def test_values_of_very_different_size_in_runs_of_many_pairs(fmt):
    """Over 31 chunks a block, some of which are done again: each gets its own result."""
    seqs, classes = many(1300, 4)
    ly = Layer(seqs, 4, 4, 64, 16, classes, fmt, seed=50)
    size = np.where(np.arange(len(ly.v)) % 61 == 0, 2.0 ** 40, 1.0)[:, None, None]
    ly.v = bf16(ly.v * size.astype(np.float32))
    t = ly.upload()
    o, lse = ly.decode(t)
    assert int(t["status"].item()) == 0
    check_attention(o, lse, ly.attention(0.125), fmt)


@pytest.mark.parametrize("room", [0, 500])
@pytest.mark.parametrize("fmt", FMTS)
def test_room_to_grow_in_the_table(room, fmt):
    """A small layer whose table array has room behind the last table: the same result, by one launch or by two."""
    ly = Layer([(256, 1), (33, 1)], 4, 2, 64, 16, [[GLOBAL, local(4, 64)]] * 2, fmt, seed=51)
    t = ly.upload()
    t["table"] = torch.cat([t["table"], torch.full((room,), -1, dtype=torch.int32, device="cuda")])
    o, lse = ly.decode(t)
    assert int(t["status"].item()) == 0
    check_attention(o, lse, ly.attention(0.125), f"{fmt} {room}")


@pytest.mark.parametrize("fmt", FMTS[1:])
def test_read_back_of_pages_that_sequences_share(fmt):
    """Sequences of one length whose tables name the same pages: each page is read back once over, the same from each."""
    ly = Layer([(90, 1), (90, 1)], 2, 1, 64, 32, [[GLOBAL]] * 2, fmt, seed=52)
    n = len(ly.table) // 2
    ly.table[n:] = ly.table[:n]
    ly.k[90:], ly.v[90:] = ly.k[:90], ly.v[:90]
    t = ly.upload(poison=False)
    ko, vo = (torch.full((ly.num_pages, 32, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sp.segpaged_pages_dequant(ly.dims(), t["ctx"], t["lq"], t["cls"], t["table"], t["offs"], t["k"], t["v"], t["scale"], ko, vo,
                              t["status"])
    want, used = ly.expected_pools()
    for got, (codes, y) in zip((ko, vo), want):
        np.testing.assert_array_equal(got.float().cpu().numpy()[used], orc.dequantise_rows(codes, y, fmt)[used])
