"""One layer's paged K/V for the decode-side tests, laid out by the oracle: page tables from its storage rule, pools
from its build, 8-bit rows from its quantiser, so that each call is tested on pools that no kernel wrote.

Tolerances of the attention (u = half a step of a type, finfo.eps / 2):
  O is rounded to bf16 once (u = 2^-8 of the value). Before that, with vmax the largest visible |V|: a probability
  rounded to fp16 (8-bit pools, u = 2^-11) or to a pair of bf16 (u = 2^-16) moves O by at most u * vmax, a sum of
  weights of 1; a logit off by d moves every weight by a factor e^+-d and so O by at most 2 d vmax (to first order),
  twice: in the weights and in their sum.
  A logit of D products in fp32 is off by at most D 2^-24 * max sum |q k| * scale, and its scaling and exponent by a few
  2^-23 of |logit|; ex2.approx is off by 2^-22. The sums over n keys are off by n 2^-24 relative at most.
  LSE is off by the logit error, the relative error of the sum, and its own rounding (2^-23 of |LSE|).
"""
import math

import numpy as np
import torch

from oracle import reference as orc

DTYPE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
GLOBAL = (1, 0, 0)


def bf16(x):
    return orc.bf16_round(np.asarray(x, np.float32))


class Layer:
    """seqs: [(L, Lq)] (Lq of the storage rule); classes: [B][Hkv] of (is_global, sink, window)."""

    def __init__(self, seqs, hq, hkv, D, P, classes, fmt, seed=0, k_scale=1.0, v_scale=1.0, spare=3):
        rng = np.random.default_rng(seed)
        self.rng, self.fmt, self.P, self.D, self.hq, self.hkv = rng, fmt, P, D, hq, hkv
        self.L = np.array([s[0] for s in seqs], np.int32)
        self.lq = np.array([s[1] for s in seqs], np.int32)
        self.B = len(seqs)
        self.cls = np.asarray(classes, np.int32).reshape(self.B, hkv, 3)
        self.cu = np.concatenate([[0], np.cumsum(self.L)]).astype(np.int32)
        n = int(self.cu[-1])
        self.k = bf16(rng.standard_normal((n, hkv, D)) * k_scale)
        self.v = bf16(rng.standard_normal((n, hkv, D)) * v_scale)
        self.q = bf16(rng.standard_normal((self.B, hq, D)))
        self.pages = [[orc.stored_logical_pages(int(self.L[b]), int(self.lq[b]), bool(c[0]), int(c[1]), int(c[2]), P)
                       for c in self.cls[b]] for b in range(self.B)]
        per = [len(p) for row in self.pages for p in row]
        self.offs = np.concatenate([[0], np.cumsum(per)]).astype(np.int32)
        self.num_pages = int(self.offs[-1]) + spare
        self.table = rng.permutation(self.num_pages)[:int(self.offs[-1])].astype(np.int32)

    # ------------------------------------------------------------------------------------------ oracle
    def expected_pools(self, k=None, v=None, rope=None):
        """[(codes or float32 values [pages, P, D], exponent bytes [pages, P] or None)] for K and V, and the mask of
        pages that some table names."""
        cu_q = np.concatenate([[0], np.cumsum(self.lq)])
        kp, vp = orc.build_pool(self.k if k is None else k, self.v if v is None else v, self.cu, cu_q, self.cls[..., 0],
                                self.cls[..., 1], self.cls[..., 2], self.P, self.table, self.offs, self.num_pages, rope)
        used = np.zeros(self.num_pages, bool)
        used[self.table] = True
        if self.fmt == "bf16":
            return [(kp, None), (vp, None)], used
        return [orc.quantise_rows(np.where(used[:, None, None], x, 0), self.fmt) for x in (kp, vp)], used

    def stored(self, x):
        """x [n, ...] (bf16 rows) as the pool's format holds them."""
        if self.fmt == "bf16":
            return x
        return orc.dequantise_rows(*orc.quantise_rows(x, self.fmt), self.fmt).astype(np.float32)

    def visible_pool_rows(self):
        """Mask [pages, P] of the pool rows some last position can see."""
        see = np.zeros((self.num_pages, self.P), bool)
        for b in range(self.B):
            for h in range(self.hkv):
                if self.L[b] == 0:
                    continue
                vis = orc.visible_keys(*(int(x) for x in self.cls[b, h]), int(self.L[b]) - 1)
                where = {lp: t for t, lp in enumerate(self.pages[b][h])}
                for lp in set((vis // self.P).tolist()):
                    rows = vis[vis // self.P == lp] % self.P
                    see[self.table[self.offs[b * self.hkv + h] + where[lp]], rows] = True
        return see

    def attention(self, scale, k=None, v=None):
        """(O [B, Hq, D], LSE [Hq, B], tolerances of both) in fp64."""
        k, v = self.stored(self.k if k is None else k), self.stored(self.v if v is None else v)
        live = [b for b in range(self.B) if self.L[b] > 0]
        o, lse = np.zeros((self.B, self.hq, self.D)), np.full((self.hq, self.B), -np.inf)
        to, tl = np.zeros_like(o), np.zeros_like(lse)
        G = self.hq // self.hkv
        for b in live:
            ks, vs = k[self.cu[b]:self.cu[b + 1]], v[self.cu[b]:self.cu[b + 1]]
            pb = orc.Problem(self.q[b:b + 1], ks, vs, np.array([0, 1], np.int32), np.array([0, self.L[b]], np.int32),
                             self.cls[b:b + 1, :, 0], self.cls[b:b + 1, :, 1], self.cls[b:b + 1, :, 2])
            ob, lb = orc.attention(pb, scale)
            o[b], lse[:, b] = ob, lb
            for h in range(self.hq):
                vis = orc.visible_keys(*(int(x) for x in self.cls[b, h // G]), int(self.L[b]) - 1)
                kk, vmax = np.abs(ks[vis, h // G]).astype(np.float64), np.abs(vs[vis, h // G]).max()
                smax = float((kk @ np.abs(self.q[b, h]).astype(np.float64)).max()) * abs(scale)
                d = (self.D + 8) * 2.0 ** -24 * smax + 2.0 ** -22
                u_p = 2.0 ** -16 if self.fmt == "bf16" else 2.0 ** -11
                tl[h, b] = d + len(vis) * 2.0 ** -24 + abs(lb[h]) * 2.0 ** -22
                to[b, h] = np.abs(ob[h]) * 2.0 ** -8 * (1 + 2.0 ** -8) + vmax * (u_p + 4 * d + 2 * len(vis) * 2.0 ** -24) + 1e-37
        return o, lse, to, tl

    # --------------------------------------------------------------------------------------------- GPU
    def upload(self, poison=True, device="cuda"):
        """dict of device tensors; poison: rows no last position sees, and pages of no table, hold NaN."""
        (kp, ky), (vp, vy) = self.expected_pools()[0]
        if poison:
            hide = ~self.visible_pool_rows()
            for pool, y in ((kp, ky), (vp, vy)):
                pool[hide] = np.nan if self.fmt == "bf16" else (0x7f if self.fmt == "e4m3" else 0x80)
                if y is not None:
                    y[hide] = 255
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(device)  # noqa: E731
        if self.fmt == "bf16":
            k, v = (torch.from_numpy(x).to(device).to(torch.bfloat16) for x in (kp, vp))
            scale = None
        else:
            k, v = (torch.from_numpy(x).to(device).view(DTYPE[self.fmt]) for x in (kp, vp))
            scale = torch.from_numpy(np.stack([ky, vy], 1).copy()).to(device)
        B, Hq = self.B, self.hq
        return {"k": k, "v": v, "scale": scale, "table": i32(self.table), "offs": i32(self.offs), "ctx": i32(self.L),
                "lq": i32(self.lq), "cls": i32(self.cls.reshape(-1)),
                "q": torch.from_numpy(self.q).to(device).to(torch.bfloat16),
                "o": torch.full((B, Hq, self.D), 7.0, dtype=torch.bfloat16, device=device),
                "lse": torch.full((Hq, B), 7.0, dtype=torch.float32, device=device),
                "status": torch.zeros(1, dtype=torch.int32, device=device)}

    def dims(self):
        from head_sparse_paged_b200 import segpaged as sp
        return sp.Dims(self.B, self.hq, self.hkv, self.D, self.P, self.num_pages)

    def workspace(self, device="cuda", fill=0xff):
        from head_sparse_paged_b200 import segpaged as sp
        return torch.full((sp.segpaged_decode_workspace_bytes(self.dims()),), fill, dtype=torch.uint8, device=device)

    def decode(self, t, scale=None, workspace=None, stream=None):
        from head_sparse_paged_b200 import segpaged as sp
        scale = 1.0 / math.sqrt(self.D) if scale is None else scale
        ws = self.workspace() if workspace is None else workspace
        sp.segpaged_attn_decode(self.dims(), t["q"], t["k"], t["v"], t["scale"], t["table"], t["offs"], t["ctx"], t["lq"],
                                t["cls"], scale, t["o"], t["lse"], ws, t["status"], stream)
        return t["o"], t["lse"]


def check_attention(o, lse, want, what=""):
    wo, wl, to, tl = want
    o, lse = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    live = np.isfinite(wl)
    assert np.array_equal(np.isneginf(lse), ~live), f"{what}: LSE of empty rows"
    eo, el = np.abs(o - wo), np.abs(np.where(live, lse, 0) - np.where(live, wl, 0))
    assert np.isfinite(o).all(), what
    assert (eo <= to).all(), f"{what}: O off by {(eo / np.maximum(to, 1e-300)).max():.2f} tolerances, {eo.max():.3e}"
    assert (el <= np.where(live, tl, 0)).all(), f"{what}: LSE off by {el.max():.3e}"


def local(S, W):
    return (0, S, W)


def shapes():
    """name -> (seqs, hq, hkv, D, P, classes): the sizes and masks where the calls can go wrong."""
    return {
        "one-token": ([(1, 1)], 2, 1, 64, 16, [[GLOBAL]]),
        "one-page-tail": ([(17, 1)], 4, 2, 64, 16, [[GLOBAL, local(0, 1)]]),
        "tiny": ([(256, 1)], 4, 2, 64, 16, [[GLOBAL, local(4, 64)]]),
        "empty-slots": ([(0, 0), (130, 1), (0, 0), (1, 1), (0, 0)], 8, 2, 128, 32,
                        [[GLOBAL, local(3, 5)]] * 5),
        "all-empty": ([(0, 0), (0, 0)], 4, 2, 128, 64, [[GLOBAL, local(3, 5)]] * 2),
        "window-one": ([(513, 1), (512, 1), (511, 1)], 8, 4, 128, 128,
                       [[local(0, 1), local(1, 1), local(300, 1), local(0, 513)]] * 3),
        "sink-meets-window": ([(700, 1), (64, 1)], 4, 4, 64, 32,
                              [[local(600, 100), local(600, 101), local(599, 100), local(900, 3)],
                               [local(64, 1), local(63, 1), local(0, 64), local(0, 65)]]),
        "odd-lengths-g16": ([(1000, 1), (77, 5), (333, 1)], 32, 2, 128, 64,
                            [[GLOBAL, local(16, 100)], [local(3, 5), GLOBAL], [local(130, 9), local(0, 200)]]),
        "mha-p128": ([(1153, 1)], 5, 5, 64, 128, [[GLOBAL, local(7, 129), local(128, 128), local(129, 255), GLOBAL]]),
        "group-128": ([(300, 1), (5, 1)], 128, 1, 128, 16, [[GLOBAL], [local(2, 2)]]),
        "group-32": ([(140, 2)], 64, 2, 64, 64, [[local(10, 33), GLOBAL]]),
        "stored-for-more": ([(900, 333), (77, 77), (600, 12)], 8, 2, 128, 64,
                            [[GLOBAL, local(16, 100)], [local(3, 5), GLOBAL], [local(300, 9), local(0, 250)]]),
        "many-pairs": ([(i * 7 % 50, min(1, i * 7 % 50)) for i in range(90)], 8, 4, 64, 16,
                       [[GLOBAL, local(2, 3), local(0, 20), local(17, 16)]] * 90),
        "one-long": ([(20011, 1)], 8, 1, 128, 64, [[GLOBAL]]),
        "long-beside-short": ([(9001, 1), (3, 1), (260, 1)], 16, 4, 128, 16,
                              [[GLOBAL, local(64, 1024), local(0, 100), local(5, 2000)]] * 3),
    }
