"""Sets a multi-layer SegPaged prefill workload up on one GPU through the C ABI and runs it.

Per layer: the storage accounting (segpaged_pages_bytes) gives every (sequence, KV head) its stored
page count, the caller-side page assignment hands out physical ids in one shared pool, segpaged_build
scatters the layer's dense K/V into the pool (with the RoPE re-alignment when the workload asks for
it), segpaged_prefill_plan produces the work units, and segpaged_attn_prefill runs the attention.
Device memory comes from PyTorch; every computation runs in libsegpaged.so.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

from . import segpaged as sp
from . import synth
from .counts import visible_counts, visible_flops  # noqa: F401  (re-exported)


@dataclass
class LayerState:
    cls: np.ndarray            # [B, Hkv, 3]
    pages_per_head: np.ndarray
    table: np.ndarray          # int32, physical ids
    offs: np.ndarray           # int32 [B*Hkv+1]
    units: np.ndarray | None = None       # plan records (work units, then combine records)
    info: dict | None = None
    table_dev: torch.Tensor | None = None
    offs_dev: torch.Tensor | None = None
    cls_dev: torch.Tensor | None = None
    units_dev: torch.Tensor | None = None
    units_host: torch.Tensor | None = None   # pinned staging copy of the plan
    upload_done: torch.cuda.Event | None = None
    q: torch.Tensor | None = None
    o: torch.Tensor | None = None
    lse: torch.Tensor | None = None
    stored_bytes: int = 0
    dense_bytes: int = 0
    k_new: torch.Tensor | None = None         # append: the query rows' keys / values [total_q, Hkv, D]
    v_new: torch.Tensor | None = None
    mass_items: np.ndarray | None = None     # token-mass plan (sparse-FFN score)
    mass_items_dev: torch.Tensor | None = None
    mass: torch.Tensor | None = None


class Runner:
    """One workload's pools, page tables, plans, queries and outputs on one device.

    shared_dense: all layers scatter the same dense K/V (drawn for layer 0) through their own tables,
    class maps and queries -- for many-layer workloads whose dense K/V would not fit in memory at once.
    keep_dense: keep each layer's dense K/V on the device after set-up (tests compare against them).
    mass: also plan and hold the per-token attention mass (the sparse-FFN score) of every layer.
    frags: gather-time RoPE fragments (frag_offs [B+1], frag_start [F], frag_cos_sin [F, D/2, 2] numpy arrays):
    the pools keep the keys as drawn and prefill and token mass re-align them per fragment as they load them.
    append: fused append-and-attend -- the build writes only the rows before each query range (the query
    rows' pool slots get unrelated values) and each prefill writes the query rows' keys/values into the pool
    while attending over them.
    graphs: run each layer's plain prefill call as a CUDA graph, captured once per plan shape, so that the
    call's launches (counter clear, prefill, combine) reach the GPU as one submission and its short launches
    do not wait on the host between them. The graph reads the same buffers as the call it was captured from,
    so every replay sees the plan, queries and pages the step has just written.
    """

    def __init__(self, w: synth.Workload, device="cuda", layers=None, keep_dense=False, page_seed_offset=0,
                 shared_dense=False, split_ctas=None, mass=False, frags=None, append=False, graphs=False):
        self.w = w
        self.device = torch.device(device)
        # long units are split across CTAs when one alone exceeds a CTA's share (short query ranges)
        self.split_ctas = (torch.cuda.get_device_properties(self.device).multi_processor_count
                           if split_ctas is None else int(split_ctas))
        self.layers = list(range(w.layers)) if layers is None else list(layers)
        self.keep_dense = keep_dense or shared_dense
        self.shared_dense = shared_dense
        self.dense = {}
        B, H = w.num_seqs, w.num_kv_heads
        self.dims = sp.Dims(B, w.num_q_heads, H, w.head_dim, w.page_size, 0)
        self.ctx = np.asarray(w.ctx_lens, np.int32)
        self.ql = np.asarray(w.q_lens, np.int32)
        self.state = {}
        base = 0
        for li in self.layers:
            cls = np.ascontiguousarray(w.classes[li], dtype=np.int32)
            stored, dense, per = sp.segpaged_pages_bytes(self.dims, self.ctx, self.ql, cls)
            table, offs, n = synth.assign_pages(per.reshape(B, H), w.page_order, seed=w.seed + 7919 * li + page_seed_offset)
            self.state[li] = LayerState(cls=cls, pages_per_head=per, table=table + base, offs=offs,
                                        stored_bytes=stored, dense_bytes=dense)
            base += n
        self.num_pages = max(base, 1)
        if w.page_order == "shuffled" and len(self.layers) > 1:   # one permutation over the whole pool
            perm = np.random.default_rng(w.seed + 104729 + page_seed_offset).permutation(self.num_pages).astype(np.int32)
            for st in self.state.values():
                st.table = perm[st.table]
        self.dims.num_pages = self.num_pages
        D, P = w.head_dim, w.page_size
        self.k_pool = torch.empty(self.num_pages, P, D, dtype=torch.bfloat16, device=self.device)
        self.v_pool = torch.empty(self.num_pages, P, D, dtype=torch.bfloat16, device=self.device)
        self.cu_k_dev = torch.from_numpy(w.cu_k()).to(self.device)
        self.ql_dev = torch.from_numpy(self.ql).to(self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.workspace = None
        self.mass_workspace = None
        self.with_mass = mass
        self.cu_q_dev = torch.from_numpy(w.cu_q().astype(np.int32)).to(self.device)
        if append and (w.rope_theta is not None or frags is not None):
            raise ValueError("append mode takes the new keys as given; it does not combine with RoPE re-alignment")
        self.append = append
        self.frags = None
        if frags is not None:
            fo, fs, fc = frags
            self.frags = (torch.from_numpy(np.ascontiguousarray(fo, dtype=np.int32)).to(self.device),
                          torch.from_numpy(np.ascontiguousarray(fs, dtype=np.int32)).to(self.device),
                          torch.from_numpy(np.ascontiguousarray(fc, dtype=np.float32)).to(self.device))
        self.rope = None
        if w.rope_theta is not None:
            self.rope = torch.from_numpy(sp.segpaged_rope_cos_sin(w.rope_theta, w.rope_deltas, D)).to(self.device)
        if self.frags is not None:
            self.rope = None          # the pools keep the keys as drawn; prefill re-aligns them per fragment
        self.scale = 1.0 / math.sqrt(D)
        # per layer: the build and plain-prefill calls with their arguments marshalled once (PreparedCall), so a
        # step's host overhead per call is one ctypes call; rebuilt when the plan's shape or the workspace changes
        self._prep_build, self._prep_prefill = {}, {}
        self.graphs = graphs
        for li in self.layers:
            self._setup_layer(li)

    # ------------------------------------------------------------------------------------ set-up
    def _setup_layer(self, li):
        w, st = self.w, self.state[li]
        st.table_dev = torch.from_numpy(st.table).to(self.device)
        st.offs_dev = torch.from_numpy(st.offs).to(self.device)
        st.cls_dev = torch.from_numpy(st.cls.reshape(-1)).to(self.device)
        if self.shared_dense:
            if not self.dense:
                _, k, v = synth.layer_inputs(w, 0, device=self.device)
                self.dense[0] = (k, v)
            q = synth.layer_inputs(w, li, device=self.device, parts="q")[0]
        else:
            q, k, v = synth.layer_inputs(w, li, device=self.device)
            if self.keep_dense:
                self.dense[li] = (k, v)
            else:
                self._tmp_dense = (k, v)
        st.q = q
        if self.append:
            k, v = self.dense_of(li)
            cq, ck = w.cu_q(), w.cu_k()
            rows = torch.cat([torch.arange(int(ck[b + 1]) - w.q_lens[b], int(ck[b + 1]), device=self.device)
                              for b in range(w.num_seqs)]) if w.total_q else torch.zeros(0, dtype=torch.long,
                                                                                          device=self.device)
            st.k_new = k[rows].contiguous()
            st.v_new = v[rows].contiguous()
        st.o = torch.empty_like(q)
        st.lse = torch.empty(w.num_q_heads, w.total_q, dtype=torch.float32, device=self.device)
        self.build_layer(li)
        self._tmp_dense = None
        self.plan_layer(li)
        st.units_dev = torch.from_numpy(np.ascontiguousarray(st.units)).to(self.device)
        st.units_host = torch.from_numpy(np.ascontiguousarray(st.units)).pin_memory()
        need = sp.segpaged_prefill_workspace_bytes(self.dims, st.info)
        if self.workspace is None or self.workspace.numel() * 4 < need:
            self.workspace = torch.zeros((need + 3) // 4, dtype=torch.int32, device=self.device)
        if self.with_mass:
            self.plan_mass(li)
            st.mass_items_dev = torch.from_numpy(np.ascontiguousarray(st.mass_items)).to(self.device)
            st.mass = torch.zeros(w.total_q, dtype=torch.float32, device=self.device)
            need = sp.segpaged_mass_workspace_bytes(self.dims, w.total_q)
            if self.mass_workspace is None or self.mass_workspace.numel() * 4 < need:
                self.mass_workspace = torch.zeros((need + 3) // 4, dtype=torch.int32, device=self.device)

    def dense_of(self, li):
        if self._tmp_dense is not None:
            return self._tmp_dense
        return self.dense[0 if self.shared_dense else li]

    _tmp_dense = None

    # -------------------------------------------------------------------------------- hot path
    def account_layer(self, li):
        """Storage accounting of one layer (host): stored and dense K+V bytes."""
        st = self.state[li]
        stored, dense, _ = sp.segpaged_pages_bytes(self.dims, self.ctx, self.ql, st.cls)
        return stored, dense

    def plan_layer(self, li):
        """Host planning of one layer's work units (SELECTVISIBLESTATE)."""
        st = self.state[li]
        plan = sp.segpaged_prefill_plan_append if self.append else sp.segpaged_prefill_plan
        st.units, st.info = plan(self.dims, self.ctx, self.ql, st.cls, st.offs, self.split_ctas)
        return st.units

    def upload_plan(self, li, stream=None):
        st = self.state[li]
        if st.upload_done is not None:
            st.upload_done.synchronize()     # the previous copy out of the staging buffer has finished
        st.units_host.numpy()[:] = st.units
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        with torch.cuda.stream(s):
            st.units_dev.copy_(st.units_host, non_blocking=True)
        st.upload_done = torch.cuda.Event()
        st.upload_done.record(s)

    def build_layer(self, li, stream=None):
        k, v = self.dense_of(li)
        st = self.state[li]
        if self.append and st.k_new is not None:
            # the pool gets unrelated (finite) values in the query rows: the fused prefill must overwrite them
            w = self.w
            ck = w.cu_k()
            k, v = k.clone(), v.clone()
            for b in range(w.num_seqs):
                lo, hi = int(ck[b + 1]) - w.q_lens[b], int(ck[b + 1])
                k[lo:hi] = -3.0 * k[lo:hi] + 1.0
                v[lo:hi] = 0.5 * v[lo:hi] - 2.0
        if self.append or self._tmp_dense is not None:       # per-call inputs: marshal them each time
            sp.segpaged_build(self.dims, k, v, self.cu_k_dev, self.ql_dev, st.cls_dev, st.table_dev, st.offs_dev,
                              self.rope, self.k_pool, self.v_pool, self.status, stream)
            return
        call = self._prep_build.get(li)
        if call is None:
            call = self._prep_build[li] = sp.prepare_build(self.dims, k, v, self.cu_k_dev, self.ql_dev, st.cls_dev,
                                                            st.table_dev, st.offs_dev, self.rope, self.k_pool,
                                                            self.v_pool, self.status)
        call(stream)

    def prefill(self, li, stream=None):
        st = self.state[li]
        if self.append:
            sp.segpaged_attn_prefill_append(self.dims, st.q, st.k_new, st.v_new, self.k_pool, self.v_pool, st.table_dev,
                                            st.units_dev, st.info, self.scale, st.o, st.lse, self.workspace,
                                            self.status, stream)
            return
        if self.frags is not None:
            sp.segpaged_attn_prefill_rope(self.dims, st.q, self.k_pool, self.v_pool, st.table_dev, st.units_dev, st.info,
                                          self.scale, *self.frags, st.o, st.lse, self.workspace, self.status, stream)
            return
        key = (id(self.workspace), tuple(st.info.values()))
        cached = self._prep_prefill.get(li)
        if cached is None or cached[0] != key:
            call = sp.prepare_attn_prefill(self.dims, st.q, self.k_pool, self.v_pool, st.table_dev, st.units_dev,
                                           st.info, self.scale, st.o, st.lse, self.workspace, self.status)
            if not self.graphs:
                cached = self._prep_prefill[li] = (key, call, None)
            else:
                call(stream)     # this call's prefill, issued directly; the graph serves the calls after it
                self._prep_prefill[li] = (key, call, capture_graph(call, self.device))
                return
        _, call, graph = cached
        if graph is None:
            call(stream)
        elif stream is None:
            graph.replay()
        else:
            with torch.cuda.stream(stream):
                graph.replay()

    def rope_realign_preferred(self) -> bool:
        """Which gather-time RoPE path the caller should take (see prefill_rope_auto): the re-alignment pass when
        some (sequence, KV head) has more than one work unit, i.e. its query range spans more than 2 x 128 / G
        positions, so that every K tile would be rotated once per unit that loads it."""
        return rope_realign_preferred(self.w.q_lens, self.w.group)

    def prefill_rope_auto(self, li, k_scratch, stream=None):
        """Prefill with the fragments' RoPE re-alignment (self.frags) by the cheaper of the two exact paths:
        segpaged_rope_realign of the layer's K pages into k_scratch (a second pool of the same shape) followed by
        the plain prefill on it, when rope_realign_preferred(); else the gather-time kernel, which rotates each K
        tile in shared memory as it lands. Both give bit-identical O and LSE."""
        st = self.state[li]
        if not self.rope_realign_preferred():
            self.prefill(li, stream)
            return "gather"
        sp.segpaged_rope_realign(self.dims, self.cu_k_dev, self.ql_dev, st.cls_dev, st.table_dev, st.offs_dev,
                                 *self.frags, self.k_pool, k_scratch, self.status, stream)
        sp.segpaged_attn_prefill(self.dims, st.q, k_scratch, self.v_pool, st.table_dev, st.units_dev, st.info,
                                 self.scale, st.o, st.lse, self.workspace, self.status, stream)
        return "realign"

    def plan_mass(self, li):
        """Host planning of one layer's token-mass items."""
        st = self.state[li]
        st.mass_items = sp.segpaged_mass_plan(self.dims, self.ctx, self.ql, st.cls, st.offs)
        return st.mass_items

    def token_mass(self, li, stream=None):
        """Attention mass each query row's token receives (needs this layer's prefill LSE)."""
        st = self.state[li]
        sp.segpaged_token_mass(self.dims, st.q, self.k_pool, st.table_dev, st.mass_items_dev, st.lse, self.scale, st.mass,
                               self.mass_workspace, self.status, stream, frags=self.frags)

    def select_topk(self, li, k_per_seq: torch.Tensor, selected: torch.Tensor, stream=None):
        """Top-k rows per sequence by this layer's mass into `selected`."""
        sp.segpaged_select_topk(self.state[li].mass, self.cu_q_dev, k_per_seq, selected, stream)

    def step(self, stream=None):
        """Prefill of every layer (pools and plans already in place)."""
        for li in self.layers:
            self.prefill(li, stream)

    def full_step(self, stream=None, on_prefill=None):
        """One pass of the whole hot path for every layer: storage accounting and planning on the host,
        the build scatter and the prefill on the device. on_prefill(li, start) brackets each prefill
        launch (start=True before, False after) for per-kernel timing."""
        for li in self.layers:
            self.account_layer(li)
            self.plan_layer(li)
            self.upload_plan(li, stream)
            self.build_layer(li, stream)
            if on_prefill:
                on_prefill(li, True)
            self.prefill(li, stream)
            if on_prefill:
                on_prefill(li, False)

    def check_status(self):
        s = int(self.status.item())
        if s:
            raise RuntimeError(f"device status word {s:#x}")


KV_DTYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


class Decoder:
    """The decode steps that follow a Runner's prefill: one new token per sequence and step, in pools of its own.

    kv: the pools' format ("bf16", "e4m3", "int8"); they are built from the runner's dense K/V (keep_dense) with
    segpaged_build or segpaged_build_quant. max_new: the most tokens a sequence grows by. Context length and query length
    are counted up together per token, so a head's page table only ever grows at its end, by a page when a sequence
    crosses a page boundary; until then a step touches nothing but the device arrays of lengths.
    graphs: replay each layer's append and attention as one CUDA graph, captured after its first direct run.
    """

    def __init__(self, r: Runner, max_new: int, kv: str = "bf16", graphs: bool = False):
        if r.append or r.frags is not None:
            raise ValueError("decoding starts from a plain runner (keys re-aligned when they are built, or not at all)")
        w = r.w
        self.r, self.w, self.max_new, self.kv, self.graphs = r, w, int(max_new), kv, graphs
        self.dtype = KV_DTYPES[kv]
        dev, B, H, D, P = r.device, w.num_seqs, w.num_kv_heads, w.head_dim, w.page_size
        self.ctx, self.ql = r.ctx.copy(), r.ql.copy()
        grow = -(-self.max_new // P) + 1                       # pages a head may need on top of its prefill's
        need = sum(int(r.state[li].pages_per_head.sum()) for li in r.layers) + len(r.layers) * B * H * grow
        self.dims = sp.Dims(B, w.num_q_heads, H, D, P, max(need, 1))
        self.free = np.random.default_rng(w.seed).permutation(self.dims.num_pages).astype(np.int32)
        self.taken = 0
        raw = torch.bfloat16 if kv == "bf16" else torch.uint8
        self.k_pool, self.v_pool = (torch.zeros(self.dims.num_pages, P, D, dtype=raw, device=dev).view(self.dtype)
                                    for _ in range(2))
        self.kv_scale = None if kv == "bf16" else torch.zeros(self.dims.num_pages, 2, P, dtype=torch.uint8, device=dev)
        self.ctx_dev = torch.from_numpy(self.ctx).to(dev)
        self.device = self.ctx_dev.device                      # with its index
        self.ql_dev = torch.from_numpy(self.ql).to(dev)
        self.cu_new = torch.arange(B + 1, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.workspaces = {}  # a layer's own (2.6 MB): steps of different layers may overlap on different streams
        self.pages, self.table_dev, self.offs_dev, self.io, self._calls = {}, {}, {}, {}, {}
        for li in r.layers:
            per = r.state[li].pages_per_head
            self.pages[li] = [list(self._take(int(n))) for n in per]
            self.table_dev[li] = torch.zeros(int(per.sum()) + B * H * grow, dtype=torch.int32, device=dev)
            self.offs_dev[li] = torch.zeros(B * H + 1, dtype=torch.int32, device=dev)
            self._upload_table(li)
            k, v = r.dense_of(li)
            cls = r.state[li].cls_dev
            build = ((sp.segpaged_build, (self.k_pool, self.v_pool)) if kv == "bf16" else
                     (sp.segpaged_build_quant, (self.k_pool, self.v_pool, self.kv_scale)))
            build[0](self.dims, k, v, r.cu_k_dev, self.ql_dev, cls, self.table_dev[li], self.offs_dev[li], r.rope, *build[1],
                     self.status)
            bf = dict(dtype=torch.bfloat16, device=dev)
            q, o = torch.zeros(B, w.num_q_heads, D, **bf), torch.zeros(B, w.num_q_heads, D, **bf)
            kn, vn = torch.zeros(B, H, D, **bf), torch.zeros(B, H, D, **bf)
            lse = torch.zeros(w.num_q_heads, B, dtype=torch.float32, device=dev)
            self.io[li] = (q, kn, vn, o, lse)
            self.workspaces[li] = torch.empty(sp.segpaged_decode_workspace_bytes(self.dims), dtype=torch.uint8, device=dev)
            seq = (self.ctx_dev, self.ql_dev, cls)
            tab = (self.table_dev[li], self.offs_dev[li])
            pools = (self.k_pool, self.v_pool, self.kv_scale)
            self._calls[li] = [sp.prepare_append(self.dims, kn, vn, self.cu_new, *seq, *tab, *pools, self.status),
                               sp.prepare_attn_decode(self.dims, q, *pools, *tab, *seq, r.scale, o, lse, self.workspaces[li],
                                                      self.status), None]

    def _take(self, n):
        ids = self.free[self.taken:self.taken + n]
        if len(ids) < n:
            raise RuntimeError("the decode pool is out of pages")
        self.taken += n
        return ids

    def _upload_table(self, li):
        flat = np.array([p for head in self.pages[li] for p in head], np.int32)
        offs = np.concatenate([[0], np.cumsum([len(head) for head in self.pages[li]])]).astype(np.int32)
        self.table_dev[li][:len(flat)].copy_(torch.from_numpy(flat))
        self.offs_dev[li].copy_(torch.from_numpy(offs))

    def advance(self):
        """Makes room for one more token per sequence; call once before the layers' steps. It changes the lengths and tables
        on the current stream, so steps that run on another stream have to be ordered against it by the caller."""
        if int(self.ctx[0] - self.r.ctx[0]) >= self.max_new:
            raise RuntimeError(f"the decoder was set up for {self.max_new} new tokens")
        self.ctx += 1
        self.ql += 1
        self.ctx_dev += 1
        self.ql_dev += 1
        if not np.any((self.ctx - 1) % self.w.page_size == 0):
            return
        for li in self.r.layers:
            per = sp.segpaged_pages_bytes(self.dims, self.ctx, self.ql, self.r.state[li].cls)[2]
            for head, n in zip(self.pages[li], per):
                head.extend(self._take(int(n) - len(head)))
            self._upload_table(li)

    def check_inputs(self, q, k_new, v_new):
        """Raises ValueError for step inputs that are not what copying them into the step's buffers would keep as it is."""
        w = self.w
        for t, heads, name in ((q, w.num_q_heads, "q"), (k_new, w.num_kv_heads, "k_new"), (v_new, w.num_kv_heads, "v_new")):
            shape = (w.num_seqs, heads, w.head_dim)
            if tuple(t.shape) != shape or t.dtype != torch.bfloat16 or t.device != self.device:
                raise ValueError(f"{name}: expected {shape} bfloat16 on {self.device}, got {tuple(t.shape)} {t.dtype} on {t.device}")

    def step(self, li, q, k_new, v_new, stream=None):
        """Layer li's attention of the new tokens: q [B, Hq, D], k_new and v_new [B, Hkv, D] bf16 (RoPE included).
        Returns O [B, Hq, D] bf16 and LSE [Hq, B], buffers that the layer's next step overwrites. With `stream`, what the
        inputs wait for has to be ordered before it by the caller; they may be freed as soon as this returns."""
        self.check_inputs(q, k_new, v_new)
        qb, kb, vb, o, lse = self.io[li]
        s = torch.cuda.current_stream(self.r.device) if stream is None else stream
        append, attend, graph = self._calls[li]
        with torch.cuda.stream(s):
            for to, t in ((qb, q), (kb, k_new), (vb, v_new)):
                to.copy_(t)
                if stream is not None:
                    t.record_stream(s)  # its memory is not given out again before the copy has run
            if graph is not None:
                graph.replay()
                return o, lse
        append(s)
        attend(s)
        if self.graphs:
            def both(st):
                append(st)
                attend(st)
            self._calls[li][2] = capture_graph(both, self.r.device)
        return o, lse

    def read_back(self, li, k_out, v_out, stream=None):
        """The layer's stored pages of an 8-bit pool as bf16 pages of the same ids (for a prefill over them)."""
        sp.segpaged_pages_dequant(self.dims, self.ctx_dev, self.ql_dev, self.r.state[li].cls_dev, self.table_dev[li],
                                  self.offs_dev[li], self.k_pool, self.v_pool, self.kv_scale, k_out, v_out, self.status,
                                  stream)

    def check_status(self):
        s = int(self.status.item())
        if s:
            raise RuntimeError(f"device status word {s:#x}")


def capture_graph(call, device) -> torch.cuda.CUDAGraph:
    """A CUDA graph of one prepared C-ABI call that has already run once on `device` (the library configures
    a kernel on its first launch on a device, which must not happen inside a capture). Capturing launches
    nothing; replaying the graph repeats the call's launches with the same arguments."""
    with torch.cuda.device(device):
        g = torch.cuda.CUDAGraph()
        # thread_local: CUDA calls other threads make meanwhile (a process group's watchdog, for one) are not
        # checked against this capture
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            call(None)
    return g


def rope_realign_preferred(q_lens, group: int) -> bool:
    """True when some sequence's query range spans more than one work unit (2 x 128 / G positions) per KV head:
    each K tile is then loaded, and rotated at gather time, by several units, and one re-alignment pass over the
    stored pages costs less."""
    return max(q_lens, default=0) > 2 * (128 // group)


def main(argv=None):
    """Sets one or more layers of a workload up and runs their prefill launches back to back (for a profiler:
    `python -m head_sparse_paged_b200.runner dsv4-flash --layers 3 --launches 2`). Layers draw their own dense
    K/V, which is freed after the build, so only the pool, the queries and the outputs stay on the device."""
    import argparse
    ap = argparse.ArgumentParser(description=main.__doc__)
    ap.add_argument("workload")
    ap.add_argument("--layers", default="0", help="comma-separated layer indices")
    ap.add_argument("--launches", type=int, default=2, help="prefill launches per layer")
    ap.add_argument("--decode", type=int, default=0, metavar="N",
                    help="decode N tokens per sequence after the prefill and print the time of a layer's step")
    ap.add_argument("--kv", choices=sorted(KV_DTYPES), default="bf16", help="format of the pools that are decoded from")
    args = ap.parse_args(argv)
    w = synth.get(args.workload)
    layers = [int(x) for x in args.layers.split(",")]
    r = Runner(w, layers=layers, keep_dense=args.decode > 0)
    torch.cuda.synchronize()
    for _ in range(args.launches):
        for li in layers:
            r.prefill(li)
    torch.cuda.synchronize()
    r.check_status()
    print(f"{w.name}: layers {layers}, {args.launches} prefill launches each, pool {r.num_pages} pages, "
          f"{torch.cuda.max_memory_allocated() / 1e9:.2f} GB peak device memory")
    if args.decode > 0:
        d = Decoder(r, args.decode, args.kv, graphs=True)
        gen = torch.Generator(device=r.device)
        gen.manual_seed(w.seed)
        new = [torch.randn(s, generator=gen, device=r.device).to(torch.bfloat16)
               for s in ((w.num_seqs, w.num_q_heads, w.head_dim), *[(w.num_seqs, w.num_kv_heads, w.head_dim)] * 2)]
        times = []
        for _ in range(args.decode):
            d.advance()
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for li in layers:
                d.step(li, *new)
            end.record()
            times.append((start, end))
        torch.cuda.synchronize()
        d.check_status()
        us = sorted(a.elapsed_time(b) * 1e3 / len(layers) for a, b in times[1:] or times)
        print(f"decode: {args.decode} tokens x {w.num_seqs} sequences from {args.kv} pools, {us[len(us) // 2]:.1f} us a layer "
              f"and step (append and attention, inputs copied in)")
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
