"""The decode-side operators on a head-sparse paged KV cache, as they are measured.

Four operators, named by a case's "op":
  decode  attention of one new token per sequence over its own stored pages (bf16, e4m3 or int8 pools)
  write   a layer's dense K/V scattered into 8-bit pages, quantised row by row on the way
  append  the new tokens' K/V written into their pages (quantised, or copied into a bf16 pool)
  read    the stored 8-bit pages read back as bf16 pages with the same ids

A row is the D values of one (token, KV head) of K or of V. An 8-bit row holds codes c and one exponent byte y, and
stands for c * 2^(y - 127): 2^(y - 127) is the smallest power of two (from 2^-126 up) that brings the row's largest
magnitude to 448 (e4m3) or 127 (int8) at most. Exponent bytes live in kv_scale [pages, 2, P] (K, then V).
"""
import math

import numpy as np
import torch

own = False

FMT_BYTES = {"bf16": 2, "e4m3": 1, "int8": 1}
FMT_DTYPE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FMT_MAX = {"e4m3": 448.0, "int8": 127.0}
MOST_TOKENS = 64 * 131072  # stored (token, KV head) rows of the largest listed case


# ------------------------------------------------------------------------------------------------ cases

def _case(op, fmt, seqs, lo, hi, hq, hkv, dim, page, n_global, sink, window, new=1):
    """seqs sequences of lo..hi tokens, hq query and hkv KV heads; n_global KV heads of each sequence keep their whole
    context, the others `sink` first and `window` last tokens; `new` appended tokens a sequence (append)."""
    return {"op": op, "fmt": fmt, "seqs": seqs, "len_lo": lo, "len_hi": hi, "q_heads": hq, "kv_heads": hkv, "dim": dim,
            "page": page, "globals": n_global, "sink": sink, "window": window, "new": new}


def listed():
    cases = {
        # the smallest layer of the workloads: a call that is all latency
        "decode-tiny-bf16": _case("decode", "bf16", 1, 256, 256, 4, 2, 64, 16, 1, 4, 64),
        # one user, an 8K context, one global head in eight
        "decode-8k-e4m3": _case("decode", "e4m3", 1, 8192, 8192, 32, 8, 128, 64, 1, 64, 1024),
        # a serving batch with ragged contexts, in each type of pool
        "decode-batch32-bf16": _case("decode", "bf16", 32, 16384, 32768, 64, 8, 128, 64, 1, 128, 2048),
        "decode-batch32-e4m3": _case("decode", "e4m3", 32, 16384, 32768, 64, 8, 128, 64, 1, 128, 2048),
        # one long context whose single global head has to be split over the whole GPU
        "decode-128k-int8": _case("decode", "int8", 1, 131071, 131071, 64, 8, 128, 128, 1, 128, 4096),
        # a layer of 64 heads with their own K/V, all of them global: the most bytes a layer has
        "decode-mha64-e4m3": _case("decode", "e4m3", 1, 131072, 131072, 64, 64, 128, 128, 64, 128, 4096),
        # a prompt's cache written once: one user; a ragged batch
        "write-8k-int8": _case("write", "int8", 1, 8192, 8192, 32, 8, 128, 64, 1, 64, 1024),
        "write-batch4-e4m3": _case("write", "e4m3", 4, 16384, 32768, 64, 8, 128, 64, 1, 128, 2048),
        # a decode step's new rows: a batch of single tokens; a few drafted tokens a sequence into bf16 pages
        "append-batch32-e4m3": _case("append", "e4m3", 32, 1025, 4099, 64, 8, 128, 64, 1, 128, 2048),
        "append-draft5-bf16": _case("append", "bf16", 7, 100, 1999, 32, 8, 128, 16, 1, 64, 1024, new=5),
        # a stored cache taken back to bf16 pages for a prefill: one user; a ragged batch
        "read-8k-int8": _case("read", "int8", 1, 8191, 8191, 32, 8, 128, 64, 1, 64, 1024),
        "read-batch4-e4m3": _case("read", "e4m3", 4, 16384, 32768, 64, 8, 128, 64, 1, 128, 2048),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "write", "append", "read"])
    fmt = rng.choice(["e4m3", "int8"] if op in ("write", "read") else ["bf16", "e4m3", "int8"])
    dim, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    hkv, group = rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice([1, 2, 4, 8, 16])
    seqs = _log_int(rng, 1, 48)
    n_global = rng.randint(0, hkv)
    sink, window = rng.randint(0, 300), _log_int(rng, 1, 5000)
    hi = _log_int(rng, 16, 131072 if op == "decode" else 32768 if op != "append" else 4096)
    # half of the largest case's rows at most, counted as if every row were kept (16 bits) or a dense source held
    hi = max(16, min(hi, MOST_TOKENS // (4 if op == "decode" else 8) // (seqs * hkv)))
    lo = rng.randint(max(1, hi // 3), hi)
    return _case(op, fmt, seqs, lo, hi, hkv * group, hkv, dim, page, n_global, sink, window,
                 new=rng.choice([1, 1, 2, rng.randint(1, 9)]) if op == "append" else 1)


def _lengths(c):
    """Context lengths of a case: spread over [len_lo, len_hi] by the golden ratio, most of them odd sizes."""
    span = c["len_hi"] - c["len_lo"]
    return [c["len_lo"] + int(span * ((b * 0.6180339887 + 0.37) % 1.0)) for b in range(c["seqs"])]


def _classes(c):
    """[seqs, kv_heads, 3] (is_global, sink, window): the global heads of sequence b start at head 3 b (mod kv_heads)."""
    B, H = c["seqs"], c["kv_heads"]
    first = 3 * np.arange(B)[:, None]
    glob = (np.arange(H)[None, :] - first) % H < c["globals"]
    cls = np.zeros((B, H, 3), np.int32)
    cls[..., 0] = glob
    cls[..., 1] = np.where(glob, 0, c["sink"])
    cls[..., 2] = np.where(glob, 0, c["window"])
    return cls


def _storage(c):
    """(pages of the sink part, first page of the window part, stored pages) of each (sequence, KV head), flat: a head
    keeps the pages of its sink tokens and of the tokens its served positions (the last `new`) can see."""
    P = c["page"]
    L = np.repeat(np.array(_lengths(c), np.int64), c["kv_heads"])
    cls = _classes(c).reshape(-1, 3).astype(np.int64)
    n_all = -(-L // P)
    ns = -(-np.minimum(cls[:, 1], L) // P)
    w0 = np.maximum(L - min(c["new"], c["len_lo"]) - cls[:, 2] + 1, 0) // P
    whole = (cls[:, 0] == 1) | (w0 <= ns)
    ns, w0 = np.where(whole, n_all, ns), np.where(whole, n_all, w0)
    return ns, w0, ns + n_all - w0


def _visible(c):
    """Visible keys of each (sequence, KV head) for its last position."""
    L = np.repeat(np.array(_lengths(c), np.int64), c["kv_heads"])
    cls = _classes(c).reshape(-1, 3).astype(np.int64)
    local = np.minimum(L, np.minimum(cls[:, 1], L) + np.minimum(cls[:, 2], L))
    return np.where(cls[:, 0] == 1, L, local)


def work(case):
    c, D, P = case, case["dim"], case["page"]
    per = FMT_BYTES[c["fmt"]] * D + (0 if c["fmt"] == "bf16" else 1)  # bytes of one stored row
    if c["op"] == "decode":
        rows, q = int(_visible(c).sum()), c["seqs"] * c["q_heads"]
        return {"bytes": 2 * rows * per + q * (4 * D + 4), "flops": 4 * D * rows * (c["q_heads"] // c["kv_heads"])}
    if c["op"] == "append":
        rows = c["seqs"] * c["kv_heads"] * min(c["new"], c["len_lo"])
        return {"bytes": 2 * rows * (2 * D + per), "flops": 0 if c["fmt"] == "bf16" else 2 * rows * 4 * D}
    rows = int(_storage(c)[2].sum()) * P
    return {"bytes": 2 * rows * (2 * D + per), "flops": 2 * rows * D * (4 if c["op"] == "write" else 1)}


# ------------------------------------------------------------------------------------------- plain forms

def _power(e):
    """2^e as float32, for whole numbers e in [-126, 127]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x, fmt):
    """(codes, exponent bytes) of rows x [..., D]."""
    x = x.float()
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)                         # top = m 2^e, m in [0.5, 1)
    # 448 = 0.875 * 2^9, 127 = 0.9921875 * 2^7
    e = e - 9 + (m > 0.875) if fmt == "e4m3" else e - 7 + (m > 0.9921875)
    e = torch.where(top == 0, -126, e).clamp(min=-126)
    y = x * _power(-e[..., None])
    codes = y.to(torch.float8_e4m3fn) if fmt == "e4m3" else y.round().to(torch.int8)
    return codes, (e + 127).to(torch.uint8)


def _values(codes, scale):
    """float32 values of rows of codes [..., D] with exponent bytes [...] (None: the codes are the values)."""
    x = codes.float()
    return x if scale is None else x * _power(scale.int()[..., None] - 127)


def _entries(s):
    """For each entry of the flat page tables: its (sequence, KV head), and the tokens of its page's rows [E, P]."""
    per = s["offs"][1:] - s["offs"][:-1]
    pair = torch.repeat_interleave(torch.arange(per.numel(), device=per.device), per.long(), output_size=s["table"].numel())
    L = s["ctx_len"].repeat_interleave(s["case"]["kv_heads"])
    sink, win, glob, P = s["cls"][:, 1], s["cls"][:, 2], s["cls"][:, 0] == 1, s["case"]["page"]
    n_all = (L + P - 1) // P
    ns = (torch.minimum(sink, L) + P - 1) // P
    w0 = (L - s["q_len"].repeat_interleave(s["case"]["kv_heads"]) - win + 1).clamp(min=0) // P
    whole = glob | (w0 <= ns)
    ns, w0 = torch.where(whole, n_all, ns), torch.where(whole, n_all, w0)
    t = torch.arange(pair.numel(), device=pair.device) - s["offs"][:-1].long()[pair]
    page = torch.where(t < ns[pair], t, w0[pair] + t - ns[pair])
    return pair, page[:, None] * P + torch.arange(P, device=pair.device), L


def _plain_decode(s):
    c = s["case"]
    B, H, D, G = c["seqs"], c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"]
    pair, tok, L = _entries(s)
    ids = s["table"].long()
    ks, vs = (None, None) if s["kv_scale"] is None else (s["kv_scale"][ids, 0], s["kv_scale"][ids, 1])
    q = s["q"].float().reshape(B * H, G, D)
    sc = torch.bmm(_values(s["k_pool"][ids], ks), q[pair].transpose(1, 2)) * s["scale"]              # [E, P, G]
    glob, sink, win = s["cls"][:, 0] == 1, s["cls"][:, 1], s["cls"][:, 2]
    see = glob[pair, None] | (tok < sink[pair, None]) | (tok >= (L - win)[pair, None])
    sc = sc.masked_fill(~(see & (tok < L[pair, None]))[..., None], float("-inf"))
    top = torch.full((B * H, G), float("-inf"), device=q.device).index_reduce(0, pair, sc.amax(1), "amax")
    p = torch.exp(sc - top[pair, None])
    total = torch.zeros(B * H, G, device=q.device).index_add(0, pair, p.sum(1))
    o = torch.zeros(B * H, G, D, device=q.device).index_add(0, pair, torch.bmm(p.transpose(1, 2), _values(s["v_pool"][ids], vs)))
    lse = (top + total.log()).reshape(B, H * G).t().contiguous()
    return [(o / total[..., None]).reshape(B, H * G, D).to(torch.bfloat16), lse]


def _as_values(pool):
    """A pool, and its exponent bytes as the powers of two they stand for."""
    return pool if pool.dtype != torch.uint8 else pool.view(torch.float8_e8m0fnu)


def _store(s, pool, which, at, rows):
    """rows [n, D] (bf16) into the pool rows `at` (page, row in the page)."""
    if s["kv_scale"] is None:
        pool[at] = rows
        return
    codes, y = _quantise(rows, s["case"]["fmt"])
    pool.view(torch.uint8)[at] = codes.view(torch.uint8)
    s["kv_scale"][at[0], which, at[1]] = y


def _plain_write(s):
    pair, tok, L = _entries(s)
    H, P = s["case"]["kv_heads"], s["case"]["page"]
    src = s["cu_k"].long()[pair // H, None] + tok
    keep = (tok < L[pair, None])[..., None]
    at = (s["table"].long()[:, None].expand(-1, P), torch.arange(P, device=tok.device).expand(tok.shape[0], P))
    src = src.clamp(max=s["k"].shape[0] - 1)
    for which, (x, pool) in enumerate(((s["k"], s["k_pool"]), (s["v"], s["v_pool"]))):
        _store(s, pool, which, at, x[src, (pair % H)[:, None]] * keep)
    return [s["k_pool"], s["v_pool"], _as_values(s["kv_scale"])]


def _plain_append(s):
    H, P = s["case"]["kv_heads"], s["case"]["page"]
    per = s["cu_new"][1:] - s["cu_new"][:-1]
    n = s["k_new"].shape[0]
    seq = torch.repeat_interleave(torch.arange(per.numel(), device=per.device), per.long(), output_size=n)
    pos = s["ctx_len"][seq] - s["cu_new"][1:][seq] + torch.arange(n, device=per.device)
    pair, tok, _ = _entries(s)
    last = s["offs"][1:].long().reshape(-1, H)[seq] - 1                                               # [n, H]: a head's last entry
    back = tok[last, 0] // P - (pos // P)[:, None]                                                    # pages before it
    at = (s["table"].long()[last - back], (pos % P)[:, None].expand(-1, H))
    _store(s, s["k_pool"], 0, at, s["k_new"])
    _store(s, s["v_pool"], 1, at, s["v_new"])
    return [s["k_pool"], s["v_pool"]] + ([] if s["kv_scale"] is None else [_as_values(s["kv_scale"])])


def _plain_read(s):
    pair, tok, L = _entries(s)
    ids = s["table"].long()
    keep = (tok < L[pair, None])[..., None]
    for which, (pool, out) in enumerate(((s["k_pool"], s["k_out"]), (s["v_pool"], s["v_out"]))):
        out[ids] = (_values(pool[ids], s["kv_scale"][ids, which]) * keep).to(torch.bfloat16)
    return [s["k_out"], s["v_out"]]


PLAIN = {"decode": _plain_decode, "write": _plain_write, "append": _plain_append, "read": _plain_read}


# ----------------------------------------------------------------------------------------- state and calls

def _rows(gen, n, D, spread):
    """n rows like a cache's: normal values, a few channels larger than the others (keys)."""
    x = torch.randn(n, D, generator=gen, device="cuda")
    if spread:
        x *= torch.exp(0.5 * torch.randn(1, D, generator=gen, device="cuda"))
    return x


def prepare(case, seed):
    c = case
    B, Hq, H, D, P = c["seqs"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1009 + 17)
    L, stored = _lengths(c), _storage(c)[2]
    new = min(c["new"], c["len_lo"])
    n_entries = int(stored.sum())
    pages = n_entries + 5  # a few pages that no table names
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    s = {
        "case": c, "scale": 1.0 / math.sqrt(D), "pages": pages,
        "table": torch.randperm(pages, generator=gen, device="cuda")[:n_entries].int(),
        "offs": i32(np.concatenate([[0], np.cumsum(stored)])),
        "ctx_len": i32(L), "q_len": i32([new] * B), "cls": i32(_classes(c).reshape(-1, 3)),
        "kv_scale": None if c["fmt"] == "bf16" else torch.zeros(pages, 2, P, dtype=torch.uint8, device="cuda"),
    }
    bf = torch.bfloat16
    s["k_pool"], s["v_pool"] = (torch.zeros(pages, P, D, dtype=FMT_DTYPE[c["fmt"]], device="cuda") for _ in range(2))
    if c["op"] != "write":  # the cache as an earlier write left it
        page, row = torch.arange(pages, device="cuda")[:, None].expand(-1, P), torch.arange(P, device="cuda").expand(pages, P)
        for which, pool in enumerate((s["k_pool"], s["v_pool"])):
            for lo in range(0, pages, 1 << 14):
                hi = min(pages, lo + (1 << 14))
                x = _rows(gen, (hi - lo) * P, D, which == 0).reshape(hi - lo, P, D).to(bf)
                _store(s, pool, which, (page[lo:hi], row[lo:hi]), x)
    if c["op"] == "decode":
        s["q"] = _rows(gen, B * Hq, D, True).reshape(B, Hq, D).to(bf)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(Hq, B, device="cuda")
    elif c["op"] == "write":
        s["cu_k"] = i32(np.concatenate([[0], np.cumsum(L)]))
        s["k"], s["v"] = (_rows(gen, sum(L) * H, D, i == 0).reshape(-1, H, D).to(bf) for i in range(2))
    elif c["op"] == "append":
        s["cu_new"] = i32(new * np.arange(B + 1))
        s["k_new"], s["v_new"] = (_rows(gen, new * B * H, D, i == 0).reshape(-1, H, D).to(bf) for i in range(2))
    else:
        s["k_out"], s["v_out"] = (torch.zeros(pages, P, D, dtype=bf, device="cuda") for _ in range(2))
    if own:
        s["call"] = _marshal(s)  # arguments checked and turned into pointers once, as a serving loop keeps them
    return s


def _marshal(s):
    """The framework's call for this state as the object a program keeps for it: it holds pointers, no results."""
    from head_sparse_paged_b200 import segpaged as sp
    c = s["case"]
    dims = sp.Dims(c["seqs"], c["q_heads"], c["kv_heads"], c["dim"], c["page"], s["pages"])
    pools = (s["k_pool"], s["v_pool"], s["kv_scale"])
    if c["op"] == "decode":
        need = sp.segpaged_decode_workspace_bytes(dims)
        s["workspace"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
        return sp.prepare_attn_decode(dims, s["q"], *pools, s["table"], s["offs"], s["ctx_len"], s["q_len"], s["cls"],
                                      s["scale"], s["o"], s["lse"], s["workspace"])
    if c["op"] == "write":
        return sp.prepare_build_quant(dims, s["k"], s["v"], s["cu_k"], s["q_len"], s["cls"], s["table"], s["offs"], None, *pools)
    if c["op"] == "append":
        return sp.prepare_append(dims, s["k_new"], s["v_new"], s["cu_new"], s["ctx_len"], s["q_len"], s["cls"], s["table"],
                                 s["offs"], *pools)
    return sp.prepare_pages_dequant(dims, s["ctx_len"], s["q_len"], s["cls"], s["table"], s["offs"], *pools, s["k_out"],
                                    s["v_out"])


def run(state):
    s = state
    if not own:
        return PLAIN[s["case"]["op"]](s)
    s["call"]()
    if s["case"]["op"] == "decode":
        return [s["o"], s["lse"]]
    if s["case"]["op"] == "read":
        return [s["k_out"], s["v_out"]]
    return [s["k_pool"], s["v_pool"]] + ([] if s["kv_scale"] is None else [_as_values(s["kv_scale"])])


# ------------------------------------------------------------------------------------------------- exact

def _power64(e):
    """2^e in 64 bits, from the exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_rows(x, fmt):
    """(values of the codes, powers of two) in 64 bits of rows x [..., D], from the rule: try every exponent in turn."""
    x = x.double()
    a = x.abs().amax(-1, keepdim=True)
    e = torch.full_like(a, -126.0)
    for k in range(-126, 128):
        e = torch.where(a > FMT_MAX[fmt] * 2.0 ** (k - 1), torch.full_like(e, float(k)), e) if k > -126 else e
    y = x * _power64(-e)
    if fmt == "int8":
        return torch.round(y), _power64(e)
    step = _power64(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)  # three bits after the leading one
    return torch.round(y / step) * step, _power64(e)


def _exact_pages(c, b, k):
    """Logical pages the storage rule keeps for (sequence, head), in order, from the tokens that need them."""
    P, L, (g, sink, win) = c["page"], _lengths(c)[b], _classes(c)[b, k].tolist()
    served = range(L - min(c["new"], c["len_lo"]), L)
    first = 0 if g else max(served[0] - win + 1, 0)
    a, w = set(range(-(-min(sink, L) // P))) if not g else set(), set(range(first // P, -(-L // P)))
    return sorted(a | w)


def exact(case, seed):
    c = case
    B, H, D, P, G = c["seqs"], c["kv_heads"], c["dim"], c["page"], c["q_heads"] // c["kv_heads"]
    if c["op"] in ("write", "read", "append") and B * H > 512:
        return None
    s = prepare(case, seed)
    offs, table = s["offs"].tolist(), s["table"].long()
    L, cls = _lengths(c), _classes(c)
    if c["op"] == "decode":
        o = torch.zeros(B, H * G, D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(H * G, B, dtype=torch.float64, device="cuda")
        for b in range(B):
            for k in range(H):
                ids = table[offs[b * H + k]:offs[b * H + k + 1]]
                pages = torch.tensor(_exact_pages(c, b, k), device="cuda")
                tok = (pages[:, None] * P + torch.arange(P, device="cuda")).reshape(-1)
                g, sink, win = cls[b, k].tolist()
                see = tok < L[b]
                if not g:
                    see &= (tok < sink) | (tok > L[b] - 1 - win)
                kv = []
                for which, pool in enumerate((s["k_pool"], s["v_pool"])):
                    x = pool[ids].double()
                    if s["kv_scale"] is not None:
                        x = x * _power64(s["kv_scale"][ids, which].long() - 127)[..., None]
                    kv.append(x.reshape(-1, D)[see])
                sc = s["q"][b, k * G:(k + 1) * G].double() @ kv[0].t() * s["scale"]
                lse[k * G:(k + 1) * G, b] = torch.logsumexp(sc, 1)
                o[b, k * G:(k + 1) * G] = torch.softmax(sc, 1) @ kv[1]
        return [o, lse]
    f64 = lambda t: t.double() if t.dtype != torch.int8 else t.clone()  # noqa: E731
    if c["op"] == "read":
        outs = [torch.zeros(s["pages"], P, D, dtype=torch.float64, device="cuda") for _ in range(2)]
        for b in range(B):
            for k in range(H):
                ids = table[offs[b * H + k]:offs[b * H + k + 1]]
                tok = torch.tensor(_exact_pages(c, b, k), device="cuda")[:, None] * P + torch.arange(P, device="cuda")
                for which, pool in enumerate((s["k_pool"], s["v_pool"])):
                    x = pool[ids].double() * _power64(s["kv_scale"][ids, which].long() - 127)[..., None]
                    outs[which][ids] = x * (tok < L[b])[..., None]
        return outs
    pools = [f64(s["k_pool"]), f64(s["v_pool"])]
    scale = None if s["kv_scale"] is None else _power64(s["kv_scale"].long() - 127)
    for b in range(B):
        for k in range(H):
            ids = table[offs[b * H + k]:offs[b * H + k + 1]]
            tok = torch.tensor(_exact_pages(c, b, k), device="cuda")[:, None] * P + torch.arange(P, device="cuda")
            lo = L[b] - min(c["new"], c["len_lo"]) if c["op"] == "append" else 0
            if c["op"] == "append":
                page, row = torch.nonzero((tok >= lo) & (tok < L[b]), as_tuple=True)
                src = int(s["cu_new"][b]) + tok[page, row] - lo
                x = (s["k_new"][src, k], s["v_new"][src, k])
            else:
                page, row = (t.reshape(-1) for t in torch.meshgrid(torch.arange(tok.shape[0], device="cuda"),
                                                                    torch.arange(P, device="cuda"), indexing="ij"))
                t = tok.reshape(-1)
                src = sum(L[:b]) + t.clamp(max=L[b] - 1)
                x = (s["k"][src, k] * (t < L[b])[:, None], s["v"][src, k] * (t < L[b])[:, None])
            for which in range(2):
                if scale is None:
                    pools[which][ids[page], row] = x[which].double()
                    continue
                codes, e = _exact_rows(x[which], c["fmt"])
                pools[which][ids[page], row] = codes.to(pools[which].dtype)
                scale[ids[page], which, row] = e[..., 0]
    return pools + ([] if scale is None else [scale])
