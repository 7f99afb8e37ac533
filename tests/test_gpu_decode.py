"""Single-token attention, the 8-bit build, append and read back on the GPU against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

from decode_common import DTYPE, GLOBAL, Layer, bf16, check_attention, local, shapes
from head_sparse_paged_b200 import segpaged as sp
from oracle import reference as orc

pytestmark = pytest.mark.gpu
FMTS = ("bf16", "e4m3", "int8")
SHAPES = shapes()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def dev_bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(torch.bfloat16)


def raw(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype != torch.bfloat16 else t.float().cpu().numpy()


def marked_pools(ly, fmt=None):
    """Pools and exponent bytes filled with a mark, to tell what a call leaves alone."""
    fmt = fmt or ly.fmt
    shape = (ly.num_pages, ly.P, ly.D)
    if fmt == "bf16":
        return torch.full(shape, 5.0, dtype=torch.bfloat16, device="cuda"), \
            torch.full(shape, 5.0, dtype=torch.bfloat16, device="cuda"), None
    k, v = (torch.full(shape, 0x33, dtype=torch.uint8, device="cuda").view(DTYPE[fmt]) for _ in range(2))
    return k, v, torch.full((ly.num_pages, 2, ly.P), 0x33, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------------------------------- 8-bit build

def _build(ly, rope=None):
    k, v, sc = marked_pools(ly)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sp.segpaged_build_quant(ly.dims(), dev_bf16(ly.k), dev_bf16(ly.v), i32(ly.cu), i32(ly.lq), i32(ly.cls.reshape(-1)),
                         i32(ly.table), i32(ly.offs), None if rope is None else torch.from_numpy(rope).cuda(), k, v, sc,
                         status)
    assert int(status.item()) == 0
    return k, v, sc


def _check_pools(ly, k, v, sc, want, used):
    """Codes and exponent bytes bit for bit; pages of no table keep their mark."""
    for which, (pool, (codes, y)) in enumerate(zip((k, v), want)):
        got, gy = raw(pool), sc.cpu().numpy()[:, which]
        np.testing.assert_array_equal(gy[used], y[used])
        zero = (codes & 127 if ly.fmt == "e4m3" else codes) == 0      # a zero's sign is not part of its value
        np.testing.assert_array_equal(np.where(zero, got & 127 if ly.fmt == "e4m3" else got, got)[used],
                                      np.where(zero, 0, codes)[used])
        assert (got[~used] == 0x33).all() and (gy[~used] == 0x33).all()


@pytest.mark.parametrize("fmt", FMTS[1:])
@pytest.mark.parametrize("name", [n for n in SHAPES if n != "all-empty"])
def test_build_quant_bit_exact(name, fmt):
    ly = Layer(*SHAPES[name], fmt, seed=3)
    want, used = ly.expected_pools()
    _check_pools(ly, *_build(ly), want, used)


@pytest.mark.parametrize("fmt", FMTS[1:])
def test_build_quant_extreme_rows(fmt):
    """Zero rows, subnormal and huge rows, magnitudes at and around a code limit, infinities and NaN."""
    ly = Layer([(96, 1)], 2, 2, 64, 32, [[GLOBAL, GLOBAL]], fmt, seed=5)
    ly.k[0] = 0
    ly.k[1] *= np.float32(2.0 ** -120)
    ly.k[2] = bf16(ly.k[2] * np.float32(2.0 ** 124))
    ly.k[3], ly.k[4], ly.k[5], ly.k[6] = 448 * 4, 450 * 4, 127.0 / 2, 127.5 / 2
    ly.k[3:7, :, 1:] *= np.float32(0.37)
    ly.k = bf16(ly.k)
    ly.v[7, 0, 3], ly.v[8, 1, 63], ly.v[9, 0, 0] = np.inf, -np.inf, np.nan
    ly.v[10] = np.float32(2.0 ** -133)
    ly.v[11] *= np.exp2(np.linspace(-40, 0, 64, dtype=np.float32))
    ly.v[11] = bf16(ly.v[11])
    want, used = ly.expected_pools()
    assert (want[1][1] == 255).sum() == 3
    _check_pools(ly, *_build(ly), want, used)


@pytest.mark.parametrize("fmt", FMTS[1:])
def test_build_quant_is_the_quantised_build(fmt):
    """With RoPE re-alignment: bit for bit the quantised form of what segpaged_build stores."""
    ly = Layer([(300, 7), (65, 65)], 4, 2, 128, 64, [[GLOBAL, local(5, 40)], [local(0, 9), GLOBAL]], fmt, seed=8)
    rope = sp.segpaged_rope_cos_sin(1e6, [1234, 77], ly.D)
    want, used = ly.expected_pools(rope=orc.rope_cos_sin(1e6, [1234, 77], ly.D))
    _check_pools(ly, *_build(ly, rope), want, used)


# ------------------------------------------------------------------------------------------------ append

def _append(ly, t, k_new, v_new, cu_new):
    sp.segpaged_append(ly.dims(), dev_bf16(k_new), dev_bf16(v_new), i32(cu_new), t["ctx"], t["lq"], t["cls"], t["table"],
                       t["offs"], t["k"], t["v"], t["scale"], t["status"])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name", ["tiny", "empty-slots", "odd-lengths-g16", "stored-for-more", "many-pairs"])
def test_append_writes_its_rows_and_no_others(name, fmt):
    ly = Layer(*SHAPES[name], fmt, seed=11)
    t = ly.upload(poison=False)
    before = [raw(t["k"]).copy(), raw(t["v"]).copy(), None if fmt == "bf16" else t["scale"].cpu().numpy().copy()]
    n = np.array([min(int(l), 1 + b % 3, int(lq)) for b, (l, lq) in enumerate(zip(ly.L, ly.lq))])
    cu = np.concatenate([[0], np.cumsum(n)]) + 2          # two rows before the first sequence, one after the last
    k_new, v_new = (bf16(ly.rng.standard_normal((int(cu[-1]) + 1, ly.hkv, ly.D)) * 3) for _ in range(2))
    _append(ly, t, k_new, v_new, cu)
    assert int(t["status"].item()) == 0
    for b in range(ly.B):
        rows = slice(int(ly.cu[b + 1]) - n[b], int(ly.cu[b + 1]))
        ly.k[rows], ly.v[rows] = k_new[cu[b]:cu[b + 1]], v_new[cu[b]:cu[b + 1]]
    want, used = ly.expected_pools()
    touched = np.zeros((ly.num_pages, ly.P), bool)
    for b in range(ly.B):
        for h in range(ly.hkv):
            for pos in range(int(ly.L[b]) - n[b], int(ly.L[b])):
                touched[ly.table[ly.offs[b * ly.hkv + h] + ly.pages[b][h].index(pos // ly.P)], pos % ly.P] = True
    for which, pool in enumerate((t["k"], t["v"])):
        got = raw(pool)
        np.testing.assert_array_equal(got[touched], want[which][0][touched])
        np.testing.assert_array_equal(got[~touched], before[which][~touched])
        if fmt != "bf16":
            gy = t["scale"].cpu().numpy()[:, which]
            np.testing.assert_array_equal(gy[touched], want[which][1][touched])
            np.testing.assert_array_equal(gy[~touched], before[2][:, which][~touched])


def test_append_drops_rows_whose_page_is_not_kept():
    """More new rows than the window's pages hold: a local head drops the ones between its sink and its window."""
    ly = Layer([(400, 1)], 2, 2, 64, 16, [[GLOBAL, local(10, 20)]], "e4m3", seed=12)
    t = ly.upload(poison=False)
    k_new, v_new = (bf16(ly.rng.standard_normal((400, 2, 64))) for _ in range(2))
    _append(ly, t, k_new, v_new, [0, 400])
    assert int(t["status"].item()) == 0
    ly.k, ly.v = k_new, v_new
    want, used = ly.expected_pools()
    for which, pool in enumerate((t["k"], t["v"])):
        row_used = used[:, None] & (t["scale"].cpu().numpy()[:, which] != 0)
        np.testing.assert_array_equal(raw(pool)[used], want[which][0][used])


# --------------------------------------------------------------------------------------------- read back

@pytest.mark.parametrize("fmt", FMTS[1:])
@pytest.mark.parametrize("name", [n for n in SHAPES if n != "all-empty"])
def test_dequant_bit_exact(name, fmt):
    ly = Layer(*SHAPES[name], fmt, seed=21)
    t = ly.upload(poison=False)
    past = np.ones((ly.num_pages, ly.P), bool)                  # rows past the context end hold NaN and read as zero
    for b in range(ly.B):
        for h in range(ly.hkv):
            for i, lp in enumerate(ly.pages[b][h]):
                past[ly.table[ly.offs[b * ly.hkv + h] + i]] = np.arange(ly.P) + lp * ly.P >= ly.L[b]
    t["scale"][torch.from_numpy(past).cuda()[:, None].expand(-1, 2, -1)] = 255
    ko, vo, _ = marked_pools(ly, "bf16")
    sp.segpaged_pages_dequant(ly.dims(), t["ctx"], t["lq"], t["cls"], t["table"], t["offs"], t["k"], t["v"], t["scale"],
                              ko, vo, t["status"])
    assert int(t["status"].item()) == 0
    want, used = ly.expected_pools()
    for out, (codes, y) in zip((ko, vo), want):
        ref = orc.dequantise_rows(codes, y, fmt)
        got = out.float().cpu().numpy()
        np.testing.assert_array_equal(got[used], np.where(past[..., None], 0, ref)[used])
        assert (got[~used] == 5.0).all()


@pytest.mark.parametrize("fmt", FMTS[1:])
def test_dequant_every_code_and_exponent(fmt):
    """All 256 codes under exponent bytes over the whole range, against fp64 rounded to bf16."""
    ly = Layer([(1024, 1)], 1, 1, 64, 128, [[GLOBAL]], fmt, seed=22)
    t = ly.upload(poison=False)
    codes = ly.rng.integers(0, 256, (ly.num_pages, ly.P, ly.D)).astype(np.uint8)
    y = (np.arange(ly.num_pages * ly.P) % 256).reshape(ly.num_pages, ly.P).astype(np.uint8)
    t["k"].view(torch.uint8).copy_(torch.from_numpy(codes))
    t["scale"][:, 0] = torch.from_numpy(y).cuda()
    ko, vo, _ = marked_pools(ly, "bf16")
    sp.segpaged_pages_dequant(ly.dims(), t["ctx"], t["lq"], t["cls"], t["table"], t["offs"], t["k"], t["v"], t["scale"],
                              ko, vo, t["status"])
    ref = torch.from_numpy(orc.dequantise_rows(codes, y, fmt)).to(torch.bfloat16).float().numpy()[ly.table]
    np.testing.assert_array_equal(ko.float().cpu().numpy()[ly.table], ref)


# -------------------------------------------------------------------------------------------- attention

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name", list(SHAPES))
def test_decode_matches_oracle_with_nan_in_every_hidden_row(name, fmt):
    ly = Layer(*SHAPES[name], fmt, seed=31)
    t = ly.upload()
    o, lse = ly.decode(t)
    assert int(t["status"].item()) == 0
    check_attention(o, lse, ly.attention(1.0 / math.sqrt(ly.D)), f"{name} {fmt}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,P,G", [(64, 16, 4), (64, 64, 16), (128, 16, 8)])
def test_decode_long_runs(D, P, G, fmt):
    """Over 2400 tiles of 128 tokens: each of 148 blocks fills its ring of stages at least twice."""
    ly = Layer([(9777, 1), (9504, 1), (9601, 1), (9473, 1)], 8 * G, 8, D, P, [[GLOBAL] * 7 + [local(33, 9000)]] * 4, fmt, seed=61)
    t = ly.upload()
    o, lse = ly.decode(t)
    assert int(t["status"].item()) == 0
    check_attention(o, lse, ly.attention(1.0 / math.sqrt(D)), f"{D} {P} {G} {fmt}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("k_scale,v_scale,scale", [(8.0, 1.0, 0.5), (1e-3, 1e3, 1.0), (2.0 ** 20, 2.0 ** -60, 2.0 ** -22),
                                                   (2.0 ** -40, 2.0 ** 60, 2.0 ** 37), (1.0, 1.0, 0.0), (1.0, 1.0, -0.3),
                                                   (1.0, 2.0 ** -114, 0.1), (1.0, 2.0 ** 122, 0.1), (100.0, 1.0, 0.09)])
def test_decode_ranges(fmt, k_scale, v_scale, scale):
    """One-hot softmaxes, uniform ones, keys and values far from 1, a negative scale."""
    ly = Layer([(777, 1), (2050, 1)], 8, 2, 128, 32, [[GLOBAL, local(20, 200)]] * 2, fmt, seed=32, k_scale=k_scale,
               v_scale=v_scale)
    o, lse = ly.decode(ly.upload(), scale=scale)
    check_attention(o, lse, ly.attention(scale), f"{fmt} {k_scale} {v_scale} {scale}")


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_rows_of_very_different_size(fmt):
    """Value rows from 2^-20 to 2^10 in one sequence: each row's own exponent counts."""
    ly = Layer([(1500, 1)], 4, 1, 64, 16, [[GLOBAL]], fmt, seed=33)
    size = np.exp2(ly.rng.uniform(-20, 10, (1500, 1, 1))).astype(np.float32)
    ly.v = bf16(ly.v * size)
    o, lse = ly.decode(ly.upload())
    check_attention(o, lse, ly.attention(0.125), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_a_visible_nan_reaches_only_its_own_heads(fmt):
    ly = Layer([(500, 1), (500, 1)], 8, 2, 64, 32, [[GLOBAL, GLOBAL]] * 2, fmt, seed=34)
    clean = ly.attention(0.125)
    ly.k[123, 1, 5] = np.nan                 # sequence 0, KV head 1: query heads 4..7
    ly.v[500 + 77, 0, 9] = np.nan            # sequence 1, KV head 0: query heads 0..3
    t = ly.upload(poison=False)
    o, lse = ly.decode(t)
    o, lse = o.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isnan(o[0, 4:]).all() and np.isnan(lse[4:, 0]).all()
    assert np.isnan(o[1, :4, 9]).all() and np.isfinite(lse[:, 1]).all()
    if fmt == "bf16":
        assert np.isfinite(np.delete(o[1, :4], 9, axis=1)).all()
    for b, hs in ((0, slice(0, 4)), (1, slice(4, 8))):
        assert (np.abs(o[b, hs] - clean[0][b, hs]) <= clean[2][b, hs]).all()
        assert (np.abs(lse[hs, b] - clean[1][hs, b]) <= clean[3][hs, b]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_is_deterministic_and_page_order_free(fmt):
    shape = SHAPES["long-beside-short"]
    a, b = Layer(*shape, fmt, seed=35), Layer(*shape, fmt, seed=35)
    b.table = np.random.default_rng(99).permutation(b.num_pages)[:len(b.table)].astype(np.int32)
    ta, tb = a.upload(), b.upload()
    first = [x.clone() for x in a.decode(ta)]
    for _ in range(3):
        for x, y in zip(a.decode(ta), first):
            assert torch.equal(x, y)
    for x, y in zip(b.decode(tb), first):
        assert torch.equal(x, y)


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_graph_replays_as_lengths_grow(fmt):
    """One captured append + decode, replayed while ctx_len, q_len, the tables and the new rows change."""
    ly = Layer([(150, 1), (63, 1)], 8, 2, 64, 16, [[GLOBAL, local(5, 40)]] * 2, fmt, seed=36)
    steps = [Layer([(150 + i, 1 + i), (63 + i, 1 + i)], 8, 2, 64, 16, [[GLOBAL, local(5, 40)]] * 2, fmt, seed=36) for i in range(20)]
    cap = len(steps[-1].table)
    n_pages = 200
    perm = np.random.default_rng(1).permutation(n_pages).astype(np.int32)
    grown = {}                                   # (sequence, head, logical page) -> physical id
    t = steps[0].upload(poison=False)
    dims = sp.Dims(2, 8, 2, 64, 16, n_pages)
    pool = (n_pages, 16, 64)
    t["k"], t["v"] = (torch.zeros(pool, dtype=DTYPE[fmt] if fmt == "bf16" else torch.uint8, device="cuda") for _ in range(2))
    if fmt != "bf16":
        t["k"], t["v"] = t["k"].view(DTYPE[fmt]), t["v"].view(DTYPE[fmt])
        t["scale"] = torch.zeros(n_pages, 2, 16, dtype=torch.uint8, device="cuda")
    t["table"] = torch.zeros(cap, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(2)
    k_all, v_all = (bf16(rng.standard_normal((2, 200, 2, 64))) for _ in range(2))
    rows_k, rows_v = (torch.zeros(400, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cu = i32([0, 0, 0])
    ws = torch.empty(sp.segpaged_decode_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    app = sp.prepare_append(dims, rows_k, rows_v, cu, t["ctx"], t["lq"], t["cls"], t["table"], t["offs"], t["k"], t["v"],
                            t["scale"], t["status"])
    dec = sp.prepare_attn_decode(dims, t["q"], t["k"], t["v"], t["scale"], t["table"], t["offs"], t["ctx"], t["lq"], t["cls"],
                                 0.125, t["o"], t["lse"], ws, t["status"])
    graph = None
    for i, st in enumerate(steps):
        table = []
        for b in range(2):
            for h in range(2):
                for lp in st.pages[b][h]:
                    if (b, h, lp) not in grown:
                        grown[b, h, lp] = perm[len(grown)]
                    table.append(grown[b, h, lp])
        new = [int(st.L[b]) if i == 0 else 1 for b in range(2)]
        t["table"][:len(table)] = i32(table)
        t["offs"].copy_(i32(st.offs))
        t["ctx"].copy_(i32(st.L))
        t["lq"].copy_(i32(st.lq))
        at = 0
        for b in range(2):
            lo, hi = int(st.L[b]) - new[b], int(st.L[b])
            rows_k[at:at + new[b]] = dev_bf16(k_all[b, lo:hi])
            rows_v[at:at + new[b]] = dev_bf16(v_all[b, lo:hi])
            at += new[b]
        cu.copy_(i32(np.concatenate([[0], np.cumsum(new)])))
        if graph is None:
            app()
            dec()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, capture_error_mode="thread_local"):
                app()
                dec()
        else:
            t["o"].fill_(9.0)
            graph.replay()
        torch.cuda.synchronize()
        assert int(t["status"].item()) == 0
        st.q = ly.q = steps[0].q
        st.k = np.concatenate([k_all[b, :st.L[b]] for b in range(2)])
        st.v = np.concatenate([v_all[b, :st.L[b]] for b in range(2)])
        check_attention(t["o"], t["lse"], st.attention(0.125), f"step {i} {fmt}")


def test_decode_on_a_side_stream():
    ly = Layer(*SHAPES["long-beside-short"], "e4m3", seed=37)
    t = ly.upload()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = ly.workspace()
    torch.cuda.synchronize()
    ly.decode(t, workspace=ws, stream=s)
    s.synchronize()
    check_attention(t["o"], t["lse"], ly.attention(1.0 / math.sqrt(ly.D)))


def test_calls_on_two_streams_with_their_own_workspaces():
    ly = [Layer(*SHAPES[n], f, seed=38) for n, f in (("one-long", "e4m3"), ("many-pairs", "bf16"))]
    ts, ws = [x.upload() for x in ly], [x.workspace() for x in ly]
    streams = [torch.cuda.Stream() for _ in ly]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, t, w, s in zip(ly, ts, ws, streams):
            x.decode(t, workspace=w, stream=s)
    torch.cuda.synchronize()
    for x, t in zip(ly, ts):
        check_attention(t["o"], t["lse"], x.attention(1.0 / math.sqrt(x.D)))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_bad_tables_set_status_and_stay_in_bounds(fmt):
    """A page id out of range, a table too short, offsets past the table: reported, and the other heads are right."""
    ly = Layer([(700, 1), (300, 1)], 8, 2, 64, 32, [[GLOBAL, local(20, 100)]] * 2, fmt, seed=39)
    want = ly.attention(0.125)
    t = ly.upload()
    t["table"][int(ly.offs[2]) + 3] = ly.num_pages + 5                     # sequence 1, KV head 0
    ly.decode(t, scale=0.125)
    assert int(t["status"].item()) == sp.STATUS_PAGE_ID
    o = t["o"].float().cpu().numpy()
    good = [(0, slice(0, 8)), (1, slice(4, 8))]
    for b, hs in good:
        assert (np.abs(o[b, hs] - want[0][b, hs]) <= want[2][b, hs]).all()
    t = ly.upload()
    t["table"] = t["table"][:-2].contiguous()                              # sequence 1, KV head 1 lacks its last pages
    ly.decode(t, scale=0.125)
    assert int(t["status"].item()) == sp.STATUS_TABLE
    o = t["o"].float().cpu().numpy()
    for b, hs in [(0, slice(0, 8)), (1, slice(0, 4))]:
        assert (np.abs(o[b, hs] - want[0][b, hs]) <= want[2][b, hs]).all()
    t = ly.upload()
    t["ctx"][0] = 764                                                      # two pages more than the tables hold
    ly.decode(t, scale=0.125)
    assert int(t["status"].item()) == sp.STATUS_TABLE
    if fmt != "bf16":
        t = ly.upload()
        t["table"][0] = -1
        ko, vo, _ = marked_pools(ly, "bf16")
        sp.segpaged_pages_dequant(ly.dims(), t["ctx"], t["lq"], t["cls"], t["table"], t["offs"], t["k"], t["v"], t["scale"],
                                  ko, vo, t["status"])
        assert int(t["status"].item()) == sp.STATUS_PAGE_ID
    t = ly.upload()
    t["table"][int(ly.offs[1]) - 1] = 1 << 30                              # sequence 0, KV head 0, its last page
    _append(ly, t, ly.k[:2], ly.v[:2], [0, 1, 2])
    assert int(t["status"].item()) == sp.STATUS_PAGE_ID
    t = ly.upload()
    _append(ly, t, bf16(np.ones((302, 2, 64))), bf16(np.ones((302, 2, 64))), [0, 1, 302])   # 301 rows, 300 tokens
    assert int(t["status"].item()) == sp.STATUS_TABLE


@pytest.mark.parametrize("fmt", FMTS)
def test_tables_inside_a_larger_array(fmt):
    """Offsets that begin past 0 and end before the table does: the entries around them belong to no head."""
    ly = Layer([(300, 7), (65, 65)], 4, 2, 64, 32, [[GLOBAL, local(5, 40)], [local(0, 9), GLOBAL]], fmt, seed=40, spare=8)
    spare = np.setdiff1d(np.arange(ly.num_pages), ly.table)[:5]
    want, used = ly.expected_pools()
    t = ly.upload(poison=False)
    inner = t["table"]
    t["table"] = i32(np.concatenate([spare[:3], ly.table, spare[3:]]))
    t["offs"] += 3
    o, lse = ly.decode(t)
    check_attention(o, lse, ly.attention(0.125), fmt)
    if fmt != "bf16":
        k, v, sc = marked_pools(ly)
        sp.segpaged_build_quant(ly.dims(), dev_bf16(ly.k), dev_bf16(ly.v), i32(ly.cu), t["lq"], t["cls"], t["table"],
                                t["offs"], None, k, v, sc, t["status"])
        _check_pools(ly, k, v, sc, want, used)
        ko, vo, _ = marked_pools(ly, "bf16")
        sp.segpaged_pages_dequant(ly.dims(), t["ctx"], t["lq"], t["cls"], t["table"], t["offs"], t["k"], t["v"], t["scale"],
                                  ko, vo, t["status"])
        assert (ko.float().cpu().numpy()[~used] == 5.0).all() and not (ko.float().cpu().numpy()[used] == 5.0).all()
    _append(ly, t, ly.k[-2:], ly.v[-2:], [0, 0, 2])                       # the rows sequence 1 already ends with
    assert int(t["status"].item()) == 0
    for which, pool in enumerate((t["k"], t["v"])):
        np.testing.assert_array_equal(raw(pool)[used], want[which][0][used])
    assert torch.equal(inner, t["table"][3:-2])


def test_two_graphs_take_turns_on_one_workspace():
    """Graphs of two different layers captured over the same workspace and replayed one after the other, in any order."""
    a, b = Layer(*SHAPES["one-long"], "e4m3", seed=41), Layer(*SHAPES["long-beside-short"], "e4m3", seed=42)
    ws = torch.full((max(len(a.workspace()), len(b.workspace())),), 0xff, dtype=torch.uint8, device="cuda")
    ts, graphs = [x.upload() for x in (a, b)], []
    for x, t in zip((a, b), ts):
        x.decode(t, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            x.decode(t, workspace=ws)
        graphs.append(g)
    for order in ((0, 1), (1, 0, 0, 1), (1, 1, 0)):
        for t in ts:
            t["o"].fill_(9.0)
            t["lse"].fill_(9.0)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for x, t in zip((a, b), ts):
            check_attention(t["o"], t["lse"], x.attention(1.0 / math.sqrt(x.D)), str(order))


@pytest.mark.parametrize("fmt", FMTS)
def test_pages_shared_by_heads_and_sequences(fmt):
    """Two sequences with the same prefix whose tables name the same pages, and one head's table used by another."""
    ly = Layer([(96, 1), (96, 1)], 4, 2, 64, 16, [[GLOBAL, GLOBAL]] * 2, fmt, seed=43)
    t = ly.upload()
    n = len(ly.table) // 4
    for other in (1, 2, 3):
        ly.table[other * n:(other + 1) * n] = ly.table[:n]
    t["table"] = i32(ly.table)
    o, lse = ly.decode(t)
    ly.k[:, 1] = ly.k[:, 0]
    ly.v[:, 1] = ly.v[:, 0]
    ly.k[96:], ly.v[96:] = ly.k[:96], ly.v[:96]
    check_attention(o, lse, ly.attention(0.125), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_lengths_that_change_between_replays_to_empty_and_back(fmt):
    """A captured call replayed with a sequence's slot emptied, filled again and the batch all empty."""
    full = [(513, 1), (40, 1), (2000, 1)]
    cls = [[GLOBAL, local(5, 100)]] * 3
    ly = Layer(full, 8, 2, 64, 32, cls, fmt, seed=44)
    t = ly.upload(poison=False)
    ws = ly.workspace()
    ly.decode(t, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="thread_local"):
        ly.decode(t, workspace=ws)
    want = ly.attention(0.125)
    per = np.diff(ly.offs).reshape(3, 2)
    flat = np.split(ly.table, ly.offs[1:-1])
    for live in ([1], [0, 1, 2], [], [2], [0, 2], [0, 1, 2]):
        keep = np.array([b in live for b in range(3)])
        t["ctx"].copy_(i32(np.where(keep, ly.L, 0)))
        t["lq"].copy_(i32(np.where(keep, ly.lq, 0)))
        t["offs"].copy_(i32(np.concatenate([[0], np.cumsum((per * keep[:, None]).reshape(-1))])))
        table = np.concatenate([flat[2 * b + h] for b in live for h in range(2)] or [np.zeros(0, np.int32)])
        t["table"][:len(table)].copy_(i32(table))
        t["o"].fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        assert int(t["status"].item()) == 0
        o, lse, to, tl = (x.copy() for x in want)
        o[~keep], lse[:, ~keep], to[~keep] = 0, -np.inf, 0
        check_attention(t["o"], t["lse"], (o, lse, to, tl), str(live))


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(fmt):
    """Page ids whose rows lie beyond 2^31 elements (and bytes) of the pools: every call, against the same pages at 0."""
    ly = Layer([(700, 3), (129, 1)], 16, 2, 128, 128, [[GLOBAL, local(20, 200)]] * 2, fmt, seed=45)
    first = (1 << 31) // (ly.P * ly.D) + 3
    t = ly.upload()
    small = {k: t[k] for k in ("k", "v", "scale")}
    dims = sp.Dims(ly.B, ly.hq, ly.hkv, ly.D, ly.P, first + ly.num_pages)

    def big(x, rows):
        out = torch.empty((dims.num_pages, *rows), dtype=x.dtype, device="cuda")
        out[first:].copy_(x)
        return out

    k, v = (big(small[x].view(torch.uint8) if fmt != "bf16" else small[x], (ly.P, ly.D)).view(small[x].dtype) for x in "kv")
    sc = None if fmt == "bf16" else big(small["scale"], (2, ly.P))
    table = t["table"] + first
    seq = (t["ctx"], t["lq"], t["cls"], table, t["offs"])
    ws = torch.empty(sp.segpaged_decode_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    sp.segpaged_attn_decode(dims, t["q"], k, v, sc, table, t["offs"], t["ctx"], t["lq"], t["cls"], 0.09, t["o"], t["lse"], ws,
                            t["status"])
    check_attention(t["o"], t["lse"], ly.attention(0.09), fmt)
    want, used = ly.expected_pools()
    sp.segpaged_append(dims, dev_bf16(ly.k[[699, 828]]), dev_bf16(ly.v[[699, 828]]), i32([0, 1, 2]), *seq, k, v, sc, t["status"])
    cut = lambda x: x.view(torch.uint8)[first:] if x.dtype != torch.bfloat16 else x[first:]  # noqa: E731
    see = ly.visible_pool_rows()
    for which, x in enumerate((k, v)):
        np.testing.assert_array_equal(raw(cut(x))[see], want[which][0][see])
    if fmt != "bf16":
        out = [torch.empty(dims.num_pages, ly.P, ly.D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        sp.segpaged_pages_dequant(dims, *seq, k, v, sc, *out, t["status"])
        for which, x in enumerate(out):
            ref = orc.dequantise_rows(*want[which], fmt)
            np.testing.assert_array_equal(x[first:].float().cpu().numpy()[see], ref[see])
        k.view(torch.uint8)[first:] = 0
        sp.segpaged_build_quant(dims, dev_bf16(ly.k), dev_bf16(ly.v), i32(ly.cu), t["lq"], t["cls"], table, t["offs"], None, k, v,
                                sc, t["status"])
        np.testing.assert_array_equal(raw(cut(k))[see] & 127, want[0][0][see] & 127)
    assert int(t["status"].item()) == 0
