"""Per-batch and per-layer drivers over the C ABI.

``ComposePlan`` owns the device copies of one batch's metadata and the plan
arrays, and builds the plan once per batch (``cpkv_plan_build``).
``ComposeLayers`` owns the writers' staging regions and the dense buffers
(two, alternated by layer parity: a dense buffer is reused two layers later)
and runs the per-layer fill + gather.  ``PagedCache`` serves from the pools:
rotated rows of new tokens into them, attention over them.  Allocation uses torch device memory;
every computation is a library kernel.
"""
from __future__ import annotations

import numpy as np
import torch

from . import cpkv


class ComposePlan:
    def __init__(self, prefix_lens, cur_lens, prefix_pages, cur_pages, writer, *, page_size: int, cp_size: int,
                 num_pool_pages: int, dense_cap_pages: int | None = None, device="cuda"):
        self.prefix_lens = np.ascontiguousarray(prefix_lens, dtype=np.int32)
        self.cur_lens = np.ascontiguousarray(cur_lens, dtype=np.int32)
        self.page_size, self.cp_size, self.num_pool_pages = page_size, cp_size, num_pool_pages
        self.T, self.C, self.D = cpkv.cpkv_plan_sizes(self.prefix_lens, self.cur_lens, page_size)
        self.dense_cap_pages = self.D if dense_cap_pages is None else int(dense_cap_pages)
        self.B = len(self.prefix_lens)
        self.device = torch.device(device)
        host_writer = np.ascontiguousarray(writer, dtype=np.int32)
        self.host_writer = host_writer
        self.d_prefix_pages = torch.as_tensor(np.ascontiguousarray(prefix_pages, dtype=np.int32)).to(self.device)
        self.d_cur_pages = torch.as_tensor(np.ascontiguousarray(cur_pages, dtype=np.int32)).to(self.device)
        self.d_writer = torch.as_tensor(host_writer).to(self.device)
        self.bufs = cpkv.plan_buffers(self.B, self.T, self.dense_cap_pages, num_pool_pages, self.device,
                                      workspace_bytes=cpkv.cpkv_plan_workspace_bytes(self.cur_lens, page_size,
                                                                                     cp_size))
        self.d_status = torch.zeros(1, dtype=torch.int32, device=self.device)

    @property
    def tokens_per_writer(self):
        """Rows each writer computes (sizes its current-row buffer)."""
        return cpkv.cpkv_writer_token_counts(self.cur_lens, self.host_writer, self.page_size, self.cp_size)

    def build(self, stream=None):
        cpkv.cpkv_plan_build(self.prefix_lens, self.cur_lens, self.d_prefix_pages, self.d_cur_pages, self.d_writer,
                             page_size=self.page_size, cp_size=self.cp_size, num_pool_pages=self.num_pool_pages,
                             dense_cap_pages=self.dense_cap_pages, out=self.bufs, d_status=self.d_status,
                             stream=stream)
        return self

    def __getitem__(self, k):
        return self.bufs[k]

    @property
    def staging_cap_pages(self) -> int:
        return self.C + 1


class ComposeLayers:
    """Staging regions (one per writer, C + 1 pages each, row 0 reserved) and
    ``num_dense`` dense buffers of ``dense_cap_pages`` pages."""

    def __init__(self, plan: ComposePlan, row_bytes: int, num_dense: int = 2):
        self.plan = plan
        self.row_bytes = row_bytes
        ps, cp = plan.page_size, plan.cp_size
        self.staging = [torch.empty((plan.staging_cap_pages * ps, row_bytes), dtype=torch.uint8, device=plan.device)
                        for _ in range(cp)]
        self.dense = [torch.empty((plan.dense_cap_pages * ps, row_bytes), dtype=torch.uint8, device=plan.device)
                      for _ in range(num_dense)]

    def fill(self, cur_rows_per_writer, stream=None, early_inputs=False, page_runs=True):
        """``early_inputs``: the rows and the plan were complete before the
        previous kernel on the stream started (cpkv.FLAG_EARLY_INPUTS).
        ``page_runs``: the plan's index arrays move each current page as one
        run (cpkv.FILL_PAGE_RUNS; they are this plan's own, so it holds)."""
        p = self.plan
        cpkv.cpkv_fill_current(p.cur_lens, cur_rows_per_writer, self.staging, page_size=p.page_size,
                               cp_size=p.cp_size, row_bytes=self.row_bytes, staging_cap_pages=p.staging_cap_pages,
                               d_staging_rows=p["staging_rows"], d_token_writer_row=p["token_writer_row"],
                               d_writer=p.d_writer, num_cur_pages=p.C, d_status=p.d_status,
                               early_inputs=early_inputs, page_runs=page_runs, stream=stream)

    def fill_planes(self, cur_planes_per_writer, plane_bytes, stream=None, early_inputs=False, page_runs=True):
        """Planar-page fill (``cur_planes_per_writer[p][w]``); the row width of
        these buffers must be ``sum(plane_bytes)``.  ``page_runs``: each plane
        of a current page moves as one run (cpkv.FILL_PAGE_RUNS)."""
        p = self.plan
        cpkv.cpkv_fill_current_planes(p.cur_lens, cur_planes_per_writer, self.staging, page_size=p.page_size,
                                      cp_size=p.cp_size, plane_bytes=plane_bytes,
                                      staging_cap_pages=p.staging_cap_pages, d_staging_rows=p["staging_rows"],
                                      d_token_writer_row=p["token_writer_row"], d_writer=p.d_writer,
                                      num_cur_pages=p.C, d_status=p.d_status, early_inputs=early_inputs,
                                      page_runs=page_runs, stream=stream)

    def gather(self, pools, dense, stream=None, consume_staging=False, early_inputs=False):
        """``pools``: the cp owner slabs [slab_pages, ps, R] of this layer.
        ``consume_staging``: the stagings are refilled before their next read,
        so their L2 lines are dropped after the gather reads them (their bytes
        are undefined afterwards).  ``early_inputs``: the plan and the pools
        were complete before the previous kernel on the stream (the fill)
        started (cpkv.GATHER_EARLY_INPUTS)."""
        if consume_staging or early_inputs:
            kinds = cpkv.GATHER_ALL | (cpkv.GATHER_CONSUME_STAGING if consume_staging else 0)
            self.gather_kinds(pools, dense, kinds | (cpkv.GATHER_EARLY_INPUTS if early_inputs else 0), stream)
            return
        p = self.plan
        table = list(pools) + list(self.staging)
        caps = [t.shape[0] for t in pools] + [p.staging_cap_pages] * p.cp_size
        cpkv.cpkv_compose_gather(table, caps, p["owner"], p["src"], dense, page_size=p.page_size,
                                 cp_size=p.cp_size, row_bytes=self.row_bytes, dense_cap_pages=p.dense_cap_pages,
                                 d_status=p.d_status, stream=stream)

    def gather_kinds(self, pools, dense, kinds, stream=None):
        """The gather restricted to slot kinds (cpkv.GATHER_*)."""
        p = self.plan
        table = list(pools) + list(self.staging)
        caps = [t.shape[0] if t is not None else 0 for t in pools] + [p.staging_cap_pages] * p.cp_size
        cpkv.cpkv_compose_gather_kinds(table, caps, p["owner"], p["src"], dense, page_size=p.page_size,
                                       cp_size=p.cp_size, row_bytes=self.row_bytes,
                                       dense_cap_pages=p.dense_cap_pages, kinds=kinds, d_status=p.d_status,
                                       stream=stream)

    def prefetch(self, pools, dense, stream=None):
        """Layer-ahead part of a compose: prefix pages and zero slots only."""
        self.gather_kinds(pools, dense, cpkv.GATHER_POOL | cpkv.GATHER_ZERO, stream)

    def consume(self, cur_rows_per_writer, dense, stream=None):
        """The rest of the layer once its current rows exist: fill, then the
        current pages only."""
        self.fill(cur_rows_per_writer, stream)
        self.gather_kinds([None] * self.plan.cp_size, dense, cpkv.GATHER_STAGING, stream)

    def compose_fused(self, pools, cur_rows_per_writer, dense, stream=None, plane_bytes=None, early_inputs=False):
        """One-pass single-GPU compose of a layer (no staging round trip); for
        planar pages, ``plane_bytes`` and ``cur_rows_per_writer[p][w]``.
        ``early_inputs``: the plan, pools and rows were complete before the
        previous kernel on the stream started (cpkv.FLAG_EARLY_INPUTS)."""
        p = self.plan
        if plane_bytes is not None:
            cpkv.cpkv_compose_fused_planes(p.cur_lens, pools, cur_rows_per_writer, p["owner"], p["src"],
                                           p["token_writer_row"], dense, page_size=p.page_size, cp_size=p.cp_size,
                                           plane_bytes=plane_bytes, dense_cap_pages=p.dense_cap_pages,
                                           d_status=p.d_status, early_inputs=early_inputs, stream=stream)
            return
        cpkv.cpkv_compose_fused(p.cur_lens, pools, cur_rows_per_writer, p["owner"], p["src"], p["token_writer_row"],
                                dense, page_size=p.page_size, cp_size=p.cp_size, row_bytes=self.row_bytes,
                                dense_cap_pages=p.dense_cap_pages, d_status=p.d_status, early_inputs=early_inputs,
                                stream=stream)

    def compose_one_launch(self, pools, cur_rows_per_writer, dense, stream=None, plane_bytes=None,
                           consume_staging=False, early_inputs=False):
        """Fill + gather of a layer in a single launch (cpkv_compose_layer; for
        planar pages, ``plane_bytes`` and ``cur_rows_per_writer[p][w]``,
        cpkv_compose_layer_planes)."""
        p = self.plan
        table = list(pools) + list(self.staging)
        caps = [t.shape[0] for t in pools] + [p.staging_cap_pages] * p.cp_size
        if plane_bytes is not None:
            cpkv.cpkv_compose_layer_planes(p.cur_lens, cur_rows_per_writer, table, caps, p["owner"], p["src"],
                                           p["token_writer_row"], dense, page_size=p.page_size, cp_size=p.cp_size,
                                           plane_bytes=plane_bytes, dense_cap_pages=p.dense_cap_pages,
                                           d_status=p.d_status, consume_staging=consume_staging,
                                           early_inputs=early_inputs, stream=stream)
            return
        cpkv.cpkv_compose_layer(p.cur_lens, cur_rows_per_writer, table, caps, p["owner"], p["src"],
                                p["token_writer_row"], dense, page_size=p.page_size, cp_size=p.cp_size,
                                row_bytes=self.row_bytes, dense_cap_pages=p.dense_cap_pages, d_status=p.d_status,
                                consume_staging=consume_staging, early_inputs=early_inputs, stream=stream)

    def compose_layer(self, layer: int, pools, cur_rows_per_writer, stream=None, consume_staging=False,
                      early_inputs=False, page_runs=True):
        """Fill + gather of one layer into the dense buffer of its parity.
        ``early_inputs``: both kernels launch early (the fill behind the
        previous kernel, the gather behind the fill); the caller promises that
        the plan, pools and rows were complete before the previous kernel on
        the stream started."""
        dense = self.dense[layer % len(self.dense)]
        self.fill(cur_rows_per_writer, stream, early_inputs=early_inputs, page_runs=page_runs)
        self.gather(pools, dense, stream, consume_staging=consume_staging, early_inputs=early_inputs)
        return dense


class PagedCache:
    """Token rows in owner pools, written and attended to by a serving step.

    ``pools``: the cp owner slabs [pages, page_size, width] of bf16 or fp16; a
    row keeps ``kv_heads`` key vectors of ``key_dim`` elements at
    ``key_offset`` and as many value vectors of ``value_dim`` at
    ``value_offset`` (elements; by default keys, then values).  ``dense``: the
    one "pool" is a composed dense buffer, whose page 0 is an ordinary page.
    The handle keeps the pools' addresses and a status word (``d_status``).
    Handles share one workspace per stream, which grows as calls need it: calls
    on a stream run one after the other, and a model has a handle per layer.
    Calls are asynchronous.  A call captured into a CUDA graph takes a
    workspace from the memory that ``torch.cuda.graph`` gives the capture,
    which belongs to the graph, so graphs may be replayed beside each other and
    beside other calls.  A ``workspace`` that the caller gives (a uint8 CUDA
    tensor of at least ``cpkv_attend_*_workspace_bytes``) is used as it is, for
    captures made by other means; calls that overlap on the GPU must not share
    one."""

    _workspaces = {}  # of all handles, by device and stream

    def __init__(self, pools, *, page_size: int, kv_heads: int, key_dim: int, value_dim: int | None = None,
                 key_offset: int = 0, value_offset: int | None = None, dense: bool = False):
        self.kv_heads, self.key_dim = int(kv_heads), int(key_dim)
        self.value_dim = self.key_dim if value_dim is None else int(value_dim)
        if value_offset is None:
            value_offset = key_offset + self.kv_heads * self.key_dim
        self.table = cpkv.PoolTable(pools, page_size, 2 * key_offset, 2 * value_offset, dense)
        self.device = self.table.device
        self.d_status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._scale = self.key_dim ** -0.5
        self._native = cpkv.serving()
        # the current stream's handle: torch's own accessor where it has one (a twentieth of current_stream())
        self._current = getattr(torch._C, "_cuda_getCurrentRawStream", None)

    def _stream(self, stream) -> int:
        if stream is not None:
            return stream if type(stream) is int else stream.cuda_stream
        if self._current is not None:
            return self._current(self.device.index)
        return torch.cuda.current_stream(self.device).cuda_stream

    def _attend(self, fn: str, args: tuple, stream: int, workspace, size):
        """Runs a call of the library, with a larger workspace where it wants one: ``size(args)`` bytes."""
        native = getattr(self._native, fn)
        mine, captured = workspace is None, False
        if mine:
            captured = self._native.captures(stream)
            if not captured:
                workspace = self._workspaces.get((self.device.index, stream))
        rc = native(*args, workspace, self.d_status, stream)
        if rc == cpkv.CPKV_ERR_CAPACITY and mine:
            with torch.cuda.device(self.device):  # the size goes by its SMs
                need = size(*args)
            if need > (0 if workspace is None else workspace.numel()):
                workspace = self._empty((need if captured else need + need // 4,), torch.uint8, stream)
                if not captured:
                    self._workspaces[self.device.index, stream] = workspace
                rc = native(*args, workspace, self.d_status, stream)
        if rc:
            cpkv._check("cpkv_" + fn, rc)

    def _empty(self, shape, dtype, stream: int):
        """Memory of the stream that the call runs on."""
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=self.device)):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def append_rotary(self, k, v, slots, positions, cos_sin, *, q=None, q_out=None, axis_of_freq=None,
                      interleaved=False, stream=None):
        """Rows of new tokens: ``k`` [tokens, kv_heads, key_dim] rotated by
        ``positions`` and ``v`` into cache rows ``slots`` (page * page_size +
        offset; negative: padding), ``q`` rotated into ``q_out`` (allocated
        when None), which is returned."""
        stream = self._stream(stream)
        if q is not None and q_out is None:
            q_out = self._empty(q.shape, q.dtype, stream)
        if axis_of_freq is not None:
            axis_of_freq = bytes(axis_of_freq)
        rc = self._native.append_rotary(self.table.native, self.kv_heads, self.key_dim, self.value_dim, k, v, slots,
                                        positions, cos_sin, self.d_status, q, q_out, axis_of_freq, interleaved, stream)
        if rc:
            cpkv._check("cpkv_append_rotary", rc)
        return q_out

    def _results(self, q, out, stream: int):
        """Where an attention's output goes."""
        if self.value_dim != self.key_dim or q.dim() != 3 or q.shape[2] != self.key_dim:
            raise cpkv.CpkvError("attend", cpkv.CPKV_ERR_ARG,
                                 "q: [tokens, heads, key_dim] over a cache of equal key and value widths")
        return self._empty(q.shape, q.dtype, stream) if out is None else out

    def attend_window(self, q, q_lens, page_table, kv_lens, *, max_kv_len: int, window: int = 0, sinks: int = 0,
                      scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
        """Causal attention of the newest ``q_lens[b]`` tokens of each request
        (None: one each) over its ``kv_lens[b]`` rows, those within ``window``
        and the first ``sinks``.  Returns ``out``; ``lse`` (float32 [tokens,
        heads]) is written when given."""
        stream = self._stream(stream)
        out = self._results(q, out, stream)
        if scale is None:
            scale = self._scale
        self._attend("attend_window", (self.table.native, self.kv_heads, q, q_lens, page_table, kv_lens, max_kv_len, window, sinks,
                                       scale, out, lse), stream, workspace, _window_bytes)
        return out

    def attend_shared(self, q, group_sizes, prefix_lens, prefix_pages, page_table, suffix_lens, *,
                      max_suffix_len: int, scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
        """A decode step of requests in consecutive groups: ``q`` [requests,
        heads, dim] over each group's shared prefix (``prefix_pages``, CSR by
        group) and each request's own ``suffix_lens[b]`` rows.  Returns
        ``out``; ``lse`` as in ``attend_window``."""
        stream = self._stream(stream)
        out = self._results(q, out, stream)
        if scale is None:
            scale = self._scale
        self._attend("attend_shared", (self.table.native, self.kv_heads, q, group_sizes, prefix_lens, prefix_pages, page_table,
                                       suffix_lens, max_suffix_len, scale, out, lse), stream, workspace, _shared_bytes)
        return out


def _window_bytes(table, kv_heads, q, q_lens, page_table, kv_lens, max_kv_len, window, sinks, *rest) -> int:
    return cpkv.cpkv_attend_window_workspace_bytes(kv_lens.shape[0], q.shape[1], kv_heads, q.shape[2], q_lens, max_kv_len, window, sinks)


def _shared_bytes(table, kv_heads, q, group_sizes, prefix_lens, prefix_pages, page_table, suffix_lens, max_suffix_len, *rest) -> int:
    return cpkv.cpkv_attend_shared_workspace_bytes(suffix_lens.shape[0], q.shape[1], kv_heads, q.shape[2], group_sizes, prefix_lens,
                                                   max_suffix_len)
