"""Decoder steps on streams of their own: inputs that are freed while their copy is still queued, layers that overlap."""
import dataclasses

import numpy as np
import pytest
import torch

from head_sparse_paged_b200 import synth
from head_sparse_paged_b200.runner import Decoder, Runner

pytestmark = pytest.mark.gpu
GLOBAL = (1, 0, 0)


def decoder(layers, kv, max_new=4, graphs=False):
    """`layers` layers of two sequences with long global heads, whose pairs are split over many blocks."""
    w = synth.custom("decoder-streams", [(9300, 64), (4000, 45)], 8, 2, 64, 16,
                     [[GLOBAL, (0, 5, 40)], [(0, 20, 16), GLOBAL]], seed=78)
    w = dataclasses.replace(w, classes=np.repeat(w.classes, layers, 0))
    r = Runner(w, layers=list(range(layers)), keep_dense=True)
    return w, Decoder(r, max_new, kv, graphs=graphs)


def inputs(w, n, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return [[torch.randn(w.num_seqs, h, w.head_dim, generator=gen, device="cuda").to(torch.bfloat16)
             for h in (w.num_q_heads, w.num_kv_heads, w.num_kv_heads)] for _ in range(n)]


@pytest.mark.parametrize("graphs", [False, True])
def test_inputs_may_be_freed_after_the_call(graphs):
    """The step waits on its stream while the inputs' memory would be given out again and overwritten."""
    w, d = decoder(1, "e4m3", graphs=graphs)
    (data,) = inputs(w, 1, 1)
    d.advance()
    o, lse = d.step(0, *data)                      # (captures the graph, if there is one)
    want = o.clone(), lse.clone()
    s = torch.cuda.Stream()
    copies = [x.clone() for x in data]
    torch.cuda.synchronize()
    for x in (o, lse):
        x.fill_(9.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    d.step(0, *copies, stream=s)
    del copies
    junk = [torch.full_like(x, 77.0) for x in data for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    del junk


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_layers_on_different_streams(kv):
    """Steps of two layers issued on two streams, many times over, against the same steps one after the other."""
    w, d = decoder(2, kv)
    data = inputs(w, 2, 2)
    d.advance()
    want = []
    for li in range(2):
        o, lse = d.step(li, *data[li])
        want.append((o.clone(), lse.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for li in range(2):
            for x in d.io[li][3:]:
                x.fill_(9.0)
        torch.cuda.synchronize()
        for s in streams:
            with torch.cuda.stream(s):
                torch.cuda._sleep(200_000)           # both are queued before either runs
        for li in range(2):
            d.step(li, *data[li], stream=streams[li])
        torch.cuda.synchronize()
        for li in range(2):
            assert torch.equal(d.io[li][3], want[li][0]) and torch.equal(d.io[li][4], want[li][1])
    d.check_status()
