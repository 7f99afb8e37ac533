"""Helper warps of single-token attention that give up: the call ends, reports SEGPAGED_STATUS_TIMEOUT, waits for no copy that
has landed already, and leaves a context in which the same call gives the right result. The waits run out by their limit
alone, which the probe library is built with (no fault, trap or hang is provoked)."""
import ctypes
import os
import subprocess
import time

import numpy as np
import pytest
import torch

from head_sparse_paged_b200 import build_ext
from head_sparse_paged_b200 import segpaged as sp

from decode_common import DTYPE

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "csrc", "decode_timeout_probe.cu")
LIB = os.path.join(HERE, "csrc", "libdecode_timeout_probe.so")


def build_probe() -> str:
    deps = [SRC] + [os.path.join(build_ext.CSRC, f) for f in build_ext.SOURCES + build_ext.HEADERS]
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(d) for d in deps):
        subprocess.check_call(["nvcc", *build_ext.NVCC_FLAGS, "-o", LIB, SRC])
    return LIB


@pytest.mark.parametrize("tries", [1, 9])
@pytest.mark.parametrize("D,P,fmt", [(128, 64, "bf16"), (128, 64, "e4m3"), (64, 16, "int8"), (64, 64, "bf16"), (128, 16, "e4m3")])
def test_helpers_that_give_up_end_the_call(D, P, fmt, tries):
    """200 tiles a block, from a few pages that all heads share. A helper without copies to issue gives up after 4
    tries (1) or after 12, with the ring of stages in its later turns (9; a try takes some 6 us). Where all four issue copies
    none may be idle that long, and the call comes to its end."""
    H, L, pages = 8, 470000, 40
    per = -(-L // P)
    dims = sp.Dims(1, 4 * H, H, D, P, pages)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(D + P)
    values = torch.randint(-8, 8, (pages, P, D), generator=gen, device="cuda")
    pool = values.to(torch.bfloat16).to(DTYPE[fmt]) if fmt != "int8" else values.to(torch.int8)
    scale = None if fmt == "bf16" else torch.full((pages, 2, P), 127, dtype=torch.uint8, device="cuda")
    table = torch.arange(H * per, device="cuda", dtype=torch.int32) % pages
    offs = torch.arange(H + 1, device="cuda", dtype=torch.int32) * per
    ctx = torch.tensor([L], dtype=torch.int32, device="cuda")
    cls = torch.tensor([1, 0, 0] * H, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 4 * H, D, dtype=torch.bfloat16, device="cuda")          # every key weighs the same
    o, lse = torch.empty_like(q), torch.empty(4 * H, 1, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(sp.segpaged_decode_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    call = sp.prepare_attn_decode(dims, q, pool, pool, scale, table, offs, ctx, None, cls, 1.0, o, lse, ws, status)
    lib = ctypes.CDLL(build_probe())
    lib.segpaged_attn_decode.restype = ctypes.c_int
    lib.segpaged_attn_decode.argtypes = sp.library().segpaged_attn_decode.argtypes
    assert lib.segpaged_test_set_idle_tries(tries) == 0
    early = sp.PreparedCall(lib.segpaged_attn_decode, "segpaged_attn_decode", call._args, call._keep)
    call()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    good = o.clone(), lse.clone()
    for _ in range(20):
        status.zero_()
        torch.cuda.synchronize()
        t0 = time.time()
        early()
        torch.cuda.synchronize()
        assert time.time() - t0 < 0.5               # a wait for a copy that has landed would take its limit of a second
        if tries == 1 and (fmt == "bf16" or (D, P) == (128, 64)):
            assert int(status.item()) == sp.STATUS_TIMEOUT
    status.zero_()
    o.fill_(9.0)
    call()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])
    full = np.bincount((torch.arange(per) % pages).numpy(), minlength=pages).astype(np.float64)   # uses of each page by head 0
    rows = values.double().cpu().numpy()
    last = L - (per - 1) * P
    total = (rows.sum(1) * full[:, None]).sum(0) - rows[(per - 1) % pages, last:].sum(0)
    want = total / L
    # half a step of bf16, and 470000 additions in fp32 of values up to 8
    assert np.abs(o[0, 0].double().cpu().numpy() - want).max() <= np.abs(want).max() * 2.0 ** -8 + 8 * L * 2.0 ** -24
    assert abs(float(lse[0, 0]) - np.log(L)) <= L * 2.0 ** -24 + 2.0 ** -18
