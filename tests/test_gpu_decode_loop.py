"""The decode-side calls as a program runs them together: a prefill's cache built (and quantised), tokens appended and
attended to step by step, the 8-bit cache read back and prefilled over -- against the fp64 oracle on the true rows."""
import numpy as np
import pytest
import torch

from decode_common import Layer, bf16, check_attention
from head_sparse_paged_b200 import segpaged as sp
from head_sparse_paged_b200 import synth
from head_sparse_paged_b200.runner import Decoder, Runner, main
from oracle import reference as orc

from gpu_common import compare

pytestmark = pytest.mark.gpu
GLOBAL = (1, 0, 0)


def workload():
    return synth.custom("decode-loop", [(200, 64), (45, 45), (16, 3)], 8, 2, 64, 16,
                        [[GLOBAL, (0, 5, 40)], [(0, 20, 16), GLOBAL], [(0, 3, 4), (0, 0, 30)]], seed=77)


def rows_of(w, r, news, upto):
    """Every sequence's K and V rows after `upto` appended tokens, in one varlen array each."""
    k, v = (x.float().cpu().numpy() for x in r.dense[0])
    cu = w.cu_k()
    return [np.concatenate([np.concatenate([x[cu[b]:cu[b + 1]], n[:upto, b]]) for b in range(w.num_seqs)])
            for x, n in ((k, news[1]), (v, news[2]))]


def as_layer(w, grown, fmt):
    return Layer([(L + grown, lq + grown) for L, lq in zip(w.ctx_lens, w.q_lens)], w.num_q_heads, w.num_kv_heads, w.head_dim,
                 w.page_size, w.classes[0], fmt)


@pytest.mark.parametrize("graphs", [False, True])
@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8"])
def test_decode_loop_matches_oracle(kv, graphs):
    w, steps = workload(), 40
    r = Runner(w, keep_dense=True)
    r.step()
    d = Decoder(r, steps, kv, graphs=graphs)
    rng = np.random.default_rng(5)
    news = [bf16(rng.standard_normal((steps, w.num_seqs, h, w.head_dim))) for h in (w.num_q_heads, 2, 2)]
    for i in range(steps):
        d.advance()
        o, lse = d.step(0, *(torch.from_numpy(n[i]).cuda().to(torch.bfloat16) for n in news))
        if i in (0, 2, 15, 16, 31, steps - 1):
            torch.cuda.synchronize()
            d.check_status()
            ly = as_layer(w, i + 1, kv)
            ly.q = news[0][i]
            ly.k, ly.v = rows_of(w, r, news, i + 1)
            check_attention(o, lse, ly.attention(r.scale), f"{kv} step {i}")
    with pytest.raises(RuntimeError, match="40 new tokens"):
        d.advance()


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_read_back_feeds_a_prefill(kv):
    """Decode 20 tokens into 8-bit pages, read them back to bf16, and prefill the last rows over the result."""
    w, steps = workload(), 20
    r = Runner(w, keep_dense=True)
    d = Decoder(r, steps, kv)
    rng = np.random.default_rng(6)
    news = [bf16(rng.standard_normal((steps, w.num_seqs, h, w.head_dim))) for h in (w.num_q_heads, 2, 2)]
    for i in range(steps):
        d.advance()
        d.step(0, *(torch.from_numpy(n[i]).cuda().to(torch.bfloat16) for n in news))
    k16, v16 = (torch.zeros(d.dims.num_pages, w.page_size, w.head_dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    d.read_back(0, k16, v16)
    offs = d.offs_dev[0].cpu().numpy()
    units, info = sp.segpaged_prefill_plan(d.dims, d.ctx, d.ql, w.classes[0], offs, 0)
    total = int(d.ql.sum())
    q = torch.randn(total, w.num_q_heads, w.head_dim, device="cuda").to(torch.bfloat16)
    o, lse = torch.empty_like(q), torch.empty(w.num_q_heads, total, device="cuda")
    ws = torch.zeros(sp.segpaged_prefill_workspace_bytes(d.dims, info), dtype=torch.uint8, device="cuda")
    sp.segpaged_attn_prefill(d.dims, q, k16, v16, d.table_dev[0], torch.from_numpy(units).cuda(), info, r.scale, o, lse, ws,
                             d.status)
    torch.cuda.synchronize()
    d.check_status()
    ly = as_layer(w, steps, kv)
    k, v = (ly.stored(x) for x in rows_of(w, r, news, steps))
    cu_q = np.concatenate([[0], np.cumsum(d.ql)]).astype(np.int32)
    c = w.classes[0]
    pb = orc.Problem(q.float().cpu().numpy(), k, v, cu_q, ly.cu, c[..., 0], c[..., 1], c[..., 2])
    o_ref, lse_ref = orc.attention(pb, r.scale)
    compare(o.float().cpu().numpy().reshape(-1, w.head_dim), lse.cpu().numpy().T.reshape(-1), o_ref, lse_ref, kv)


def test_decode_equals_a_prefill_of_one_query():
    """The same bf16 pool, tables laid out for one query: the decode call against segpaged_attn_prefill."""
    w = synth.llama_70b_decode(3, 1)
    r = Runner(w)
    r.step()
    st = r.state[0]
    o, lse = torch.empty_like(st.q), torch.empty_like(st.lse)
    ws = torch.empty(sp.segpaged_decode_workspace_bytes(r.dims), dtype=torch.uint8, device="cuda")
    ctx = torch.from_numpy(r.ctx).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sp.segpaged_attn_decode(r.dims, st.q, r.k_pool, r.v_pool, None, st.table_dev, st.offs_dev, ctx, None, st.cls_dev, r.scale,
                            o, lse, ws, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    # both are within their own bounds of the exact result: bf16 outputs and, in the prefill, bf16 probabilities
    v = float(r.v_pool.float().abs().max())
    assert (o.float() - st.o.float()).abs().max().item() <= v * (2 * 2.0 ** -8 + 2.0 ** -8)
    assert (lse - st.lse).abs().max().item() <= 1e-3


def test_runner_command_decodes(capsys):
    assert main(["tiny", "--decode", "3", "--kv", "int8"]) == 0
    assert "decode: 3 tokens x 1 sequences from int8 pools" in capsys.readouterr().out
