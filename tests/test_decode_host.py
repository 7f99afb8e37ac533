"""Host side of the decode-side calls (refusals, the binding's checks) and pins of the oracle's 8-bit rows. No GPU."""
import ctypes

import numpy as np
import pytest
import torch

from decode_common import GLOBAL, Layer, local, shapes
from head_sparse_paged_b200 import segpaged as sp
from oracle import reference as orc


# -------------------------------------------------------------------------------------- the oracle's rows

def test_e4m3_table_matches_torch():
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(orc.e4m3_values(), got)


def test_e4m3_rounding_matches_torch_on_ties_and_random_values():
    mags = orc.e4m3_values()[:127]
    mids = (mags[1:] + mags[:-1]) / 2
    y = np.concatenate([mags, mids, np.nextafter(mids.astype(np.float32), 0).astype(np.float64),
                        np.random.default_rng(0).uniform(0, 448, 5000)])
    y = np.concatenate([y, -y]).astype(np.float32).astype(np.float64)
    got = orc.e4m3_values()[orc._nearest_e4m3(y)]
    np.testing.assert_array_equal(got, torch.from_numpy(y).float().to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("fmt,limit", [("e4m3", 448.0), ("int8", 127.0)])
def test_row_exponent_is_the_smallest_that_fits(fmt, limit):
    for top, e in ((limit, 0), (np.nextafter(limit, 1e9), 1), (limit * 2.0 ** -9, -9), (limit * 2.0 ** 100, 100),
                   (0.0, -126), (2.0 ** -133, -126), (limit * 2.0 ** -126, -126), (limit * 2.0 ** -125, -125)):
        codes, y = orc.quantise_rows(np.array([[top, -top / 2, 0.0, top / 4]]), fmt)
        assert int(y[0]) - 127 == e, (top, y)
        step = 2.0 ** e * (32 if fmt == "e4m3" else 1)
        assert abs(orc.dequantise_rows(codes, y, fmt)[0, 0] - top) <= step / 2
    assert orc.quantise_rows(np.array([[1.0, np.inf], [np.nan, 0.0], [1.0, 2.0]]), fmt)[1].tolist()[:2] == [255, 255]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_quantised_rows_are_within_half_a_step(fmt):
    x = orc.bf16_round(np.random.default_rng(1).standard_normal((400, 64)).astype(np.float32) *
                       np.exp2(np.random.default_rng(2).uniform(-30, 30, (400, 1))).astype(np.float32))
    codes, y = orc.quantise_rows(x, fmt)
    back, scale = orc.dequantise_rows(codes, y, fmt), 2.0 ** (y.astype(np.float64) - 127)[:, None]
    half = np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10) if fmt == "e4m3" else 0.5 * scale
    assert (np.abs(back - x) <= half).all()


@pytest.mark.parametrize("name", list(shapes()))
def test_every_visible_key_is_in_a_stored_page(name):
    """The decode's keys (last position) lie in the pages the storage rule keeps, for every shape the GPU tests use."""
    ly = Layer(*shapes()[name], "bf16")
    per = sp.segpaged_pages_bytes(ly.dims(), ly.L, ly.lq, ly.cls)[2]
    np.testing.assert_array_equal(per, np.diff(ly.offs))
    for b in range(ly.B):
        for h in range(ly.hkv):
            if ly.L[b]:
                vis = orc.visible_keys(*(int(x) for x in ly.cls[b, h]), int(ly.L[b]) - 1)
                assert set((vis // ly.P).tolist()) <= set(ly.pages[b][h])


# ------------------------------------------------------------------------------------------------ refusals

OK, NULL, DIMS, CAPACITY, ALIGN, FORMAT = 0, -1, -2, -6, -8, -10
P16, P8 = 4096, 4104          # pointer values that are only compared, never read: every call below is refused first


def _call(name, dims=None, **change):
    """The C call `name` with plausible arguments, `change` replacing some: refused before any device work."""
    d = (dims or sp.Dims(2, 8, 2, 64, 16, 10)).c()
    order = {
        "segpaged_build_quant": ["fmt", "k_dense", "v_dense", "cu_k", "q_len", "cls", "table", "tlen", "offs", "rope", "k", "v",
                                 "sc", "status", "stream"],
        "segpaged_append": ["fmt", "k_new", "v_new", "n", "cu", "ctx", "q_len", "cls", "table", "tlen", "offs", "k", "v", "sc",
                            "status", "stream"],
        "segpaged_pages_dequant": ["fmt", "ctx", "q_len", "cls", "table", "tlen", "offs", "k", "v", "sc", "ko", "vo", "status",
                                   "stream"],
        "segpaged_attn_decode": ["fmt", "q", "k", "v", "sc", "table", "tlen", "offs", "ctx", "q_len", "cls", "scale", "o",
                                 "lse", "ws", "ws_bytes", "status", "stream"],
    }[name]
    default = {"fmt": 1, "n": 3, "tlen": 8, "scale": 0.125, "ws_bytes": 1 << 40, "rope": None, "status": None, "stream": None}
    args = [change.get(a, default.get(a, P16)) for a in order]
    return getattr(sp.library(), name)(None if change.get("no_dims") else ctypes.byref(d), *args)


NAMES = ("segpaged_build_quant", "segpaged_append", "segpaged_pages_dequant", "segpaged_attn_decode")


@pytest.mark.parametrize("name", NAMES)
def test_refusals_shared(name):
    assert _call(name, no_dims=True) == NULL
    for bad in (sp.Dims(2, 8, 2, 96, 16, 10), sp.Dims(2, 8, 3, 64, 16, 10), sp.Dims(2, 6, 2, 64, 16, 10),
                sp.Dims(2, 8, 2, 64, 24, 10), sp.Dims(-1, 8, 2, 64, 16, 10), sp.Dims(2, 8, 2, 64, 16, 0),
                sp.Dims(2, 8, 2, 64, 16, -1), sp.Dims(2 ** 30, 8, 2, 64, 16, 10)):
        assert _call(name, bad) == DIMS, bad
    assert _call(name, fmt=3) == FORMAT and _call(name, fmt=-1) == FORMAT
    for a in ("k", "v", "sc"):
        assert _call(name, **{a: None}) == NULL
        assert _call(name, **{a: P8}) == ALIGN
    for a in ("cls", "offs", "table"):
        assert _call(name, **{a: None}) == NULL
    assert _call(name, sp.Dims(0, 8, 2, 64, 16, 10)) == OK           # no sequences: nothing to do


@pytest.mark.parametrize("name", ["segpaged_build_quant", "segpaged_pages_dequant"])
def test_8bit_only_calls_refuse_bf16_pools(name):
    assert _call(name, fmt=0) == FORMAT


def test_refusals_of_each_call():
    for a in ("k_dense", "v_dense", "cu_k", "q_len"):
        assert _call("segpaged_build_quant", **{a: None}) == NULL
    for a in ("k_dense", "v_dense", "rope"):
        assert _call("segpaged_build_quant", **{a: P8}) == ALIGN
    for a in ("k_new", "v_new", "cu", "ctx"):
        assert _call("segpaged_append", **{a: None}) == NULL
    assert _call("segpaged_append", k_new=P8) == ALIGN and _call("segpaged_append", v_new=P8) == ALIGN
    assert _call("segpaged_append", n=-1) == DIMS and _call("segpaged_append", tlen=-1) == DIMS
    assert _call("segpaged_append", n=0) == OK
    for a in ("ctx", "ko", "vo"):
        assert _call("segpaged_pages_dequant", **{a: None}) == NULL
    assert _call("segpaged_pages_dequant", ko=P8) == ALIGN and _call("segpaged_pages_dequant", tlen=-1) == DIMS
    for a in ("q", "ctx", "o", "lse", "ws"):
        assert _call("segpaged_attn_decode", **{a: None}) == NULL
    for a in ("q", "o", "ws"):
        assert _call("segpaged_attn_decode", **{a: P8}) == ALIGN
    for bad in (float("nan"), float("inf")):
        assert _call("segpaged_attn_decode", scale=bad) == DIMS
    for bad in (2.9e38, -2.9e38):                            # finite, but not times log2(e)
        assert _call("segpaged_attn_decode", scale=bad) == DIMS
    assert _call("segpaged_attn_decode", ws_bytes=16) == CAPACITY and _call("segpaged_attn_decode", tlen=-1) == DIMS
    assert sp.error_string(FORMAT).startswith("a pool format")


class _Fake:
    """A stand-in for a CUDA tensor, as far as the binding looks at one."""
    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, shape, dtype, contiguous=True):
        self.shape, self.dtype, self._c = tuple(shape), dtype, contiguous

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return 1

    def is_contiguous(self):
        return self._c

    def data_ptr(self):
        return 4096


def test_binding_refuses_mismatched_tensors(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    dims = sp.Dims(2, 8, 2, 64, 16, 10)
    i32, bf, f8, u8 = torch.int32, torch.bfloat16, torch.float8_e4m3fn, torch.uint8
    good = dict(q=_Fake((2, 8, 64), bf), k_pool=_Fake((10, 16, 64), f8), v_pool=_Fake((10, 16, 64), f8),
                kv_scale=_Fake((10, 2, 16), u8), page_table=_Fake((8,), i32), page_table_offs=_Fake((5,), i32),
                ctx_len=_Fake((2,), i32), q_len=None, cls=_Fake((12,), i32), softmax_scale=0.1, o=_Fake((2, 8, 64), bf),
                lse=_Fake((8, 2), torch.float32), workspace=_Fake((1 << 20,), u8))
    call = sp.prepare_attn_decode(dims, **good)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)         # made for cuda:0, used while cuda:1 is current
    with pytest.raises(ValueError, match="prepared on cuda:0"):
        call()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    bad = dict(q=_Fake((2, 7, 64), bf), k_pool=_Fake((10, 16, 64), torch.float16), v_pool=_Fake((10, 16, 64), torch.int8),
               kv_scale=_Fake((10, 16), u8), page_table=_Fake((8,), torch.int64), page_table_offs=_Fake((4,), i32),
               ctx_len=_Fake((1,), i32), q_len=_Fake((1,), i32), cls=_Fake((11,), i32), o=_Fake((2, 8, 64), torch.float16),
               lse=_Fake((15,), torch.float32))
    for key, t in bad.items():
        with pytest.raises(ValueError):
            sp.prepare_attn_decode(dims, **{**good, key: t})
    with pytest.raises(ValueError):
        sp.prepare_attn_decode(dims, **{**good, "kv_scale": None})
    with pytest.raises(ValueError, match="contiguous"):
        sp.prepare_attn_decode(dims, **{**good, "q": _Fake((2, 8, 64), bf, contiguous=False)})
    new = dict(k_new=_Fake((3, 2, 64), bf), v_new=_Fake((3, 2, 64), bf), cu_seqlens_new=_Fake((3,), i32),
               ctx_len=good["ctx_len"], q_len=None, cls=good["cls"], page_table=good["page_table"],
               page_table_offs=good["page_table_offs"], k_pool=good["k_pool"], v_pool=good["v_pool"], kv_scale=good["kv_scale"])
    sp.prepare_append(dims, **new)
    for key, t in dict(k_new=_Fake((3, 64, 2), bf), v_new=_Fake((2, 2, 64), bf), cu_seqlens_new=_Fake((2,), i32)).items():
        with pytest.raises(ValueError):
            sp.prepare_append(dims, **{**new, key: t})
    with pytest.raises(ValueError):
        sp.prepare_pages_dequant(dims, good["ctx_len"], None, good["cls"], good["page_table"], good["page_table_offs"],
                                 good["k_pool"], good["v_pool"], good["kv_scale"], _Fake((9, 16, 64), bf),
                                 _Fake((10, 16, 64), bf))


@pytest.mark.parametrize("name", NAMES)
def test_more_heads_than_the_kernels_can_index_are_refused(name):
    """(sequence, KV head) pairs are counted in 32 bits, three class values each."""
    assert _call(name, sp.Dims(400_000_000, 2, 2, 64, 16, 10)) == DIMS


def test_more_tiles_than_the_attention_can_count_are_refused():
    """Half tiles of all passes over the tables, and six for the end of each pair, are counted in 32 bits."""
    for dims, tlen in ((sp.Dims(1, 8, 8, 64, 16, 10), 1 << 31), (sp.Dims(1, 8, 8, 64, 16, 10), 1 << 40),
                       (sp.Dims(1, 128, 1, 64, 16, 10), 1 << 28), (sp.Dims(700_000_000, 1, 1, 64, 16, 10), 1 << 28)):
        assert _call("segpaged_attn_decode", dims, tlen=tlen) == DIMS, (dims, tlen)
