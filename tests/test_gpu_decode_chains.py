"""Decode-side calls that read what the call right before them wrote, on one stream with nothing in between: each launch may
start while the one before it still runs, and has to see all of what that one wrote."""
import math

import numpy as np
import pytest
import torch

from decode_common import GLOBAL, Layer, bf16, check_attention, local
from head_sparse_paged_b200 import segpaged as sp
from oracle import reference as orc

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(torch.bfloat16)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def layer(fmt, seed):
    return Layer([(3000, 5), (777, 1), (64, 64), (1, 1)], 16, 2, 128, 64, [[GLOBAL, local(70, 500)]] * 4, fmt, seed=seed)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_builds_and_read_backs_in_turn(fmt, graph):
    """Two contexts written to the same pages in turn, each read back right behind: every read back is of its own write."""
    a, b = layer(fmt, 1), layer(fmt, 2)
    b.table = a.table
    t = a.upload(poison=False)
    dense = [(dev(x.k), dev(x.v)) for x in (a, b)]
    out = [[torch.zeros(a.num_pages, a.P, a.D, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    cu = i32(a.cu)
    build = [sp.prepare_build_quant(a.dims(), k, v, cu, t["lq"], t["cls"], t["table"], t["offs"], None, t["k"], t["v"],
                                    t["scale"], t["status"]) for k, v in dense]
    read = [sp.prepare_pages_dequant(a.dims(), t["ctx"], t["lq"], t["cls"], t["table"], t["offs"], t["k"], t["v"], t["scale"],
                                     ko, vo, t["status"]) for ko, vo in out]

    def both():
        for x, y in zip(build, read):
            x()
            y()
    both()
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            both()
    for _ in range(25):
        for pair in out:
            for x in pair:
                x.fill_(7.0)
        g.replay() if graph else both()
    torch.cuda.synchronize()
    assert int(t["status"].item()) == 0
    for ly, (ko, vo) in zip((a, b), out):
        want, used = ly.expected_pools()
        for got, (codes, y) in zip((ko, vo), want):
            ref = orc.dequantise_rows(codes, y, fmt)
            np.testing.assert_array_equal(got.float().cpu().numpy()[used], ref[used])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_appends_and_read_backs_in_turn(fmt):
    """The last rows of each sequence overwritten 20 times, read back into buffers of their own after each."""
    ly = layer(fmt, 3)
    t = ly.upload(poison=False)
    cu = i32(np.arange(5))
    rng = np.random.default_rng(4)
    rows = [(bf16(rng.standard_normal((4, 2, 128)) * 2.0 ** i), bf16(rng.standard_normal((4, 2, 128)))) for i in range(20)]
    new = [(dev(k), dev(v)) for k, v in rows]
    kn, vn = torch.zeros_like(new[0][0]), torch.zeros_like(new[0][0])
    out = [[torch.zeros(ly.num_pages, ly.P, ly.D, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in rows]
    torch.cuda.synchronize()
    for (k, v), (ko, vo) in zip(new, out):
        kn.copy_(k)
        vn.copy_(v)
        sp.segpaged_append(ly.dims(), kn, vn, cu, t["ctx"], t["lq"], t["cls"], t["table"], t["offs"], t["k"], t["v"], t["scale"],
                           t["status"])
        sp.segpaged_pages_dequant(ly.dims(), t["ctx"], t["lq"], t["cls"], t["table"], t["offs"], t["k"], t["v"], t["scale"], ko,
                                  vo, t["status"])
    torch.cuda.synchronize()
    assert int(t["status"].item()) == 0
    last = ly.cu[1:] - 1
    for (k, v), pair in zip(rows, out):
        ly.k[last], ly.v[last] = k, v
        want, used = ly.expected_pools()
        for got, (codes, y) in zip(pair, want):
            np.testing.assert_array_equal(got.float().cpu().numpy()[used], orc.dequantise_rows(codes, y, fmt)[used])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
def test_appends_and_attention_in_turn(fmt):
    """Each attention sees the rows, the lengths and the tables that were written right before it."""
    ly = layer(fmt, 5)
    t = ly.upload(poison=False)
    cu = i32(np.arange(5))
    rng = np.random.default_rng(6)
    rows = [(bf16(rng.standard_normal((4, 2, 128)) * 3), bf16(rng.standard_normal((4, 2, 128)))) for _ in range(12)]
    new = [(dev(k), dev(v)) for k, v in rows]
    table, ws, res = t["table"], ly.workspace(), []
    t["table"] = torch.zeros_like(table)
    torch.cuda.synchronize()
    for k, v in new:
        t["table"].copy_(table)
        sp.segpaged_append(ly.dims(), k, v, cu, t["ctx"], t["lq"], t["cls"], t["table"], t["offs"], t["k"], t["v"], t["scale"],
                           t["status"])
        o, lse = ly.decode(t, workspace=ws)
        res.append((o.clone(), lse.clone()))
        t["o"].fill_(9.0)
        t["table"].fill_(0)
    torch.cuda.synchronize()
    assert int(t["status"].item()) == 0
    last = ly.cu[1:] - 1
    for i, ((k, v), (o, lse)) in enumerate(zip(rows, res)):
        ly.k[last], ly.v[last] = k, v
        if i in (0, 1, 10, 11):
            check_attention(o, lse, ly.attention(1 / math.sqrt(128)), f"{fmt} {i}")
