"""B200 partitioned attention with selective attention-state reuse.

The token sequence is split into P context partitions; for every (query
partition, KV partition) pair -- or, with KV groups, every (query partition,
group of adjacent KV partitions) unit -- the plan either recomputes the
attention state (output, log-sum-exp) or reuses the one cached at the
previous denoising step, and the states of each query partition are composed
by an exact log-sum-exp merge (DiTango: "Cost-Effective Parallel Diffusion
Generation with Selective Attention State Reuse").  A cache can be merged
into coarser groups without recomputation to shrink it.  An optional
frame-tile mask keeps only some frame tiles (Efficient-vDiT: "Efficient Video
Diffusion Transformers With Attention Tile").

Beside the states, a history of keys and values can be kept in 4 bits
(KV4Cache), and attention can be restricted, per head and block of queries, to
the key blocks that a cheap score selects (BlockSparseAttention); both give
states of the same kind.

All compute runs in libditango.so (CUDA, sm_100a) through its C ABI
(include/ditango.h); this package only marshals arguments.  PyTorch is used
for device memory and streams.
"""
from __future__ import annotations

from . import _abi
from ._abi import (  # noqa: F401
    DitangoError, Geometry, PLAN_FRESH, PLAN_REUSE, PLAN_SKIP, LIB_PATH, EXPORTED,
    ditango_version, ditango_check_geom, ditango_num_active, ditango_state_rows,
    ditango_slot_table, ditango_plan_workspace_size, ditango_plan, ditango_attn_partial,
    ditango_merge, ditango_cache_update, ditango_set_wait_limit_ns,
    ditango_selftest_bounded_wait, ditango_plan_noalloc, ditango_cache_compose, status_string,
    ditango_plan_error, error_state, ditango_plan_from_mass, ditango_checked_build,
    ditango_check_status, PAGE, QBLOCK, kv4, ditango_block_tables, ditango_kv4_write,
    ditango_kv4_read, ditango_kv4_summary, ditango_kv4_attn, ditango_kv4_attn_workspace_size,
    ditango_kv4_select, ditango_block_summary, ditango_block_summaries, ditango_block_select,
    ditango_block_attn,
)


def check_tensor(t, name, shape, dtypes, contiguous=False):
    """Raise unless t is a tensor of one of `dtypes` with this shape, on a
    CUDA device, its last dimension contiguous (the whole tensor when
    `contiguous`).  The kernels see raw addresses and strides only, so these
    are checked here, before anything is launched."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: a torch.Tensor is required, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be on a CUDA device, is on {t.device}")


class PartitionedAttention:
    """Device buffers for one geometry and the three-call step.

    The state buffer (O [slots, B*H, Lmax, d] float32, or bfloat16 with
    state_bf16=True, a compressed cache; lse float32 [slots, B*H, Lmax]) is
    the attention-state cache: a step writes its fresh states into their
    slots and the merge reads every active unit from it, so after a step the
    cache holds this step's fresh states and the reused ones.  The merge also
    leaves the next plan's mass score in the workspace, so the next plan does
    not read the cache again; code that writes the cache tensors directly
    must set mass_from_merge = False.  group_off
    (partition offsets of the KV groups) makes the units (query partition,
    KV group); None keeps one group per partition.
    """

    def __init__(self, B, H, N, d, part_off, frame_off=None, frame_mask=None,
                 device="cuda", strides=None, state_bf16=False, group_off=None):
        import torch
        self.B, self.H, self.N, self.d = B, H, N, d
        self.part_off = list(part_off)
        self.frame_off = None if frame_off is None else list(frame_off)
        self.frame_mask = frame_mask
        self.group_off = None if group_off is None else list(group_off)
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"the state cache lives on a CUDA device, not {self.device}")
        self.geom = self._geometry(strides)
        self.P = self.geom.P
        self.G = self.geom.G
        self.n_slots = ditango_num_active(self.geom)
        self.Lmax = ditango_state_rows(self.geom)
        BH = B * H
        dev = self.device
        self.state_bf16 = bool(state_bf16)
        self.state_O = torch.empty((self.n_slots, BH, self.Lmax, d),
                                   dtype=torch.bfloat16 if self.state_bf16 else torch.float32,
                                   device=dev)
        self.state_lse = torch.empty((self.n_slots, BH, self.Lmax), dtype=torch.float32, device=dev)
        self.valid = torch.zeros(self.n_slots, dtype=torch.uint8, device=dev)
        self.plan = torch.zeros(self.P * self.G, dtype=torch.int8, device=dev)
        self.fresh_list = torch.zeros(max(self.n_slots, 1), dtype=torch.int32, device=dev)
        self.counts = torch.zeros(2, dtype=torch.int32, device=dev)
        self.score = torch.zeros(self.P * self.G, dtype=torch.float32, device=dev)
        self.ws_bytes = ditango_plan_workspace_size(self.geom)
        self.workspace = torch.empty(max(self.ws_bytes, 16), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        # the attention kernel's work counter (each launch leaves it at zero)
        self.work_counter = torch.zeros(2, dtype=torch.int32, device=dev)
        # the workspace holds the mass partials of the last merge, and the
        # cache has not changed since: the next plan need not read the cache
        self.mass_from_merge = False

    def _geometry(self, strides):
        s = strides or (None, None, None)
        return Geometry(self.B, self.H, self.N, self.d, self.part_off, self.frame_off,
                        self.frame_mask, q_strides=s[0], k_strides=s[1], v_strides=s[2],
                        group_off=self.group_off)

    def check_inputs(self, Q, K, V, out=None, out_lse=None):
        """Shapes, dtypes and devices of a step's tensors (raises on a mismatch)."""
        import torch
        qkv = (self.B, self.H, self.N, self.d)
        for name, t in (("Q", Q), ("K", K), ("V", V)):
            check_tensor(t, name, qkv, (torch.bfloat16,))
        if out is not None:
            check_tensor(out, "out", qkv, (torch.float32, torch.bfloat16))
        if out_lse is not None:
            check_tensor(out_lse, "out_lse", (self.B, self.H, self.N), (torch.float32,),
                         contiguous=True)

    def _bind(self, Q, K, V):
        want = tuple(tuple(t.stride()[:3]) for t in (Q, K, V))
        have = (tuple(self.geom.g.q_strides), tuple(self.geom.g.k_strides), tuple(self.geom.g.v_strides))
        if want != have:
            self.geom = self._geometry(want)

    def plan_step(self, band_k=0, budget=1.0, anchor=False, stream=None):
        """The plan of the next attention call.  After a merge (which left the
        mass score of the states it composed in the workspace) the selection
        runs alone; otherwise the mass score is read from the cache."""
        if not anchor and self.mass_from_merge:
            ditango_plan_from_mass(self.geom, self.workspace, self.ws_bytes, self.valid, band_k,
                                   budget, self.plan, self.fresh_list, self.counts, self.score,
                                   stream)
        else:
            ditango_plan(self.geom, None if anchor else self.state_lse, self.valid, band_k, budget,
                         anchor, self.plan, self.fresh_list, self.counts, self.score,
                         self.workspace, self.ws_bytes, stream)
        self.mass_from_merge = False

    def partial(self, Q, K, V, scale=0.0, stream=None, drift_rows=None):
        import torch
        self.check_inputs(Q, K, V)
        if drift_rows is not None:
            check_tensor(drift_rows, "drift_rows", (self.P, self.B * self.H, self.Lmax),
                         (torch.float32,), contiguous=True)
        self._bind(Q, K, V)
        self.mass_from_merge = False
        ditango_attn_partial(self.geom, Q, K, V, self.fresh_list, self.counts, scale,
                             self.state_O, self.state_lse, 1, self.valid, self.status, stream,
                             state_bf16=self.state_bf16, drift_rows=drift_rows,
                             work_counter=self.work_counter)

    def merge(self, out, out_lse=None, stream=None):
        import torch
        qkv = (self.B, self.H, self.N, self.d)
        check_tensor(out, "out", qkv, (torch.float32, torch.bfloat16))
        if out_lse is not None:
            check_tensor(out_lse, "out_lse", (self.B, self.H, self.N), (torch.float32,),
                         contiguous=True)
        ditango_merge(self.geom, self.plan, None, None, self.state_O, self.state_lse, self.valid, 0,
                      out, out.dtype == torch.float32, tuple(out.stride()[:3]), out_lse, stream,
                      state_bf16=self.state_bf16, mass_partials=self.workspace)
        self.mass_from_merge = True

    def step(self, Q, K, V, out, out_lse=None, band_k=0, budget=1.0, anchor=False, scale=0.0,
             stream=None):
        """plan -> partial attention of the fresh units -> merge, on one stream."""
        self.check_inputs(Q, K, V, out, out_lse)
        self.plan_step(band_k, budget, anchor, stream)
        self.partial(Q, K, V, scale, stream)
        self.merge(out, out_lse, stream)

    def compose(self, group_off, stream=None):
        """A new PartitionedAttention with coarser KV groups whose cache is this
        cache's states merged group by group (no attention is recomputed).
        Every boundary of group_off must be one of this object's boundaries.
        The caller may drop this object afterwards to free the finer cache."""
        coarse = PartitionedAttention(self.B, self.H, self.N, self.d, self.part_off, self.frame_off,
                                      self.frame_mask, self.device, None, self.state_bf16,
                                      group_off)
        ditango_cache_compose(self.geom, coarse.geom, self.state_O, self.state_lse, self.valid,
                              coarse.state_O, coarse.state_lse, coarse.valid, self.state_bf16,
                              stream)
        return coarse


class ErrorPlanner:
    """Anchor-guided, error-growth planning of a PartitionedAttention's steps
    (DiTango, 1. Anchor-Guided Selection Planner).

    Step 0 and every anchor_every-th step after it are anchor steps (every
    active unit fresh).  The step after an anchor recomputes the importance w
    from the cache; the others hold it.  Between anchors each unit's
    predicted reuse error w * (age + delta_i) ranks the non-band units under
    the budget, delta_i being the local state's drift that the attention
    call of the previous step measured.  The schedule is host logic; every
    number is computed on the device.
    """

    def __init__(self, pa, band_k, budget, anchor_every):
        import torch
        if anchor_every < 1:
            raise ValueError("anchor_every must be >= 1")
        self.pa = pa
        self.band_k, self.budget, self.anchor_every = band_k, budget, anchor_every
        dev = pa.device
        self.w = torch.zeros(pa.P * pa.G, dtype=torch.float32, device=dev)
        self.age = torch.zeros(max(pa.n_slots, 1), dtype=torch.float32, device=dev)
        self.delta = torch.zeros(pa.P, dtype=torch.float32, device=dev)
        self.local_ok = torch.zeros(pa.P, dtype=torch.uint8, device=dev)
        self.drift_rows = torch.zeros((pa.P, pa.B * pa.H, pa.Lmax), dtype=torch.float32, device=dev)
        self.es = error_state(self.w, self.age, self.delta, self.local_ok, self.drift_rows)
        self.step_index = 0

    def is_anchor(self, s):
        return s % self.anchor_every == 0

    def plan(self, stream=None):
        s = self.step_index
        pa = self.pa
        ditango_plan_error(pa.geom, pa.state_lse, pa.valid, self.band_k, self.budget,
                           self.is_anchor(s), s > 0 and self.is_anchor(s - 1), self.es, pa.plan,
                           pa.fresh_list, pa.counts, pa.score, pa.workspace, pa.ws_bytes, stream)

    def step(self, Q, K, V, out, out_lse=None, scale=0.0, stream=None):
        """plan by predicted error -> attention of the fresh units (measuring the
        local drift) -> merge."""
        self.pa.check_inputs(Q, K, V, out, out_lse)    # before the plan advances the ages
        self.plan(stream)
        self.pa.partial(Q, K, V, scale, stream, drift_rows=self.drift_rows)
        self.pa.merge(out, out_lse, stream)
        self.step_index += 1


class _Launcher:
    """Calls into the library for one device.  The calls of the objects below
    take a few microseconds on the device, so this is the short way to them:
    plain addresses, stride arrays made once, the device and its current stream
    looked up without the objects around them."""

    def __init__(self, device):
        import torch
        self.index = device.index
        self._current, self._guard = torch.cuda.current_device, torch.cuda.device
        self._raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._arrays = {}

    def strides(self, t, n):
        """The first n strides of t as a host array (kept: a program has few)."""
        key = t.stride()
        got = self._arrays.get((key, n))
        if got is None:
            if len(self._arrays) > 256:
                self._arrays.clear()
            got = self._arrays[key, n] = _abi._i64s(key[:n])
        return got

    def __call__(self, name, stream, *args):
        """Library function `name` on args (addresses and numbers) and the stream,
        which comes last; launches on this device whatever the current one is."""
        if self._current() != self.index:
            with self._guard(self.index):
                st = getattr(_abi._lib, name)(*args, _abi._stream(stream))
        elif stream is None and self._raw is not None:
            st = getattr(_abi._lib, name)(*args, self._raw(self.index))
        else:
            st = getattr(_abi._lib, name)(*args, _abi._stream(stream))
        if st:
            raise DitangoError(name, st)


def _addr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, shape, dtypes, device, contiguous=False):
    """check_tensor, and the device the buffers are on.  One pass over the
    properties in the common case (these calls take a few microseconds on the
    device); what is wrong is found and said by check_tensor."""
    try:
        if (t.dtype in dtypes and t.shape == shape and t.device == device
                and (t.is_contiguous() or not contiguous and (shape[-1] == 1 or t.stride(-1) == 1))):
            return
    except AttributeError:
        pass
    check_tensor(t, name, shape, dtypes, contiguous)
    raise ValueError(f"{name}: on {t.device}, the buffers are on {device}")


def _lse(t, shape, device):
    """A float32 tensor of this shape and any strides."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
        raise TypeError("out_lse: a float32 tensor is required")
    if t.shape != shape or t.device != device:
        raise ValueError(f"out_lse: a tensor of shape {tuple(shape)} on {device} is required")


def _width(lists):
    """The last dimension of lists, whose length the caller chooses (at least 1)."""
    shape = getattr(lists, "shape", ())
    return max(shape[-1], 1) if len(shape) else 1


class KV4Cache:
    """A paged history of keys and values in 4 bits, and attention over it.

    Holds the pages (data, uint8 [n_pages, Hkv, 64 * (d + 8)]), the tables of
    up to max_requests requests of up to max_blocks pages each (block_table,
    kv_len, q_off), the slots of up to max_tokens new tokens (slot_map) and the
    page summaries (sum_codes, sum_scale).  A step of a batch is

        cache.tables(ctx_len, new_len, free_pages)   # place the new tokens
        cache.write(K, V)                            # K, V [T, Hkv, d] bf16
        cache.summarize(ctx_len)                     # only if select() is used
        sel, count = cache.select(Q, k)              # only for single tokens
        cache.attend(Q, out, out_lse, ...)           # Q [T, H, d] bf16

    Every length stays on the device; nothing synchronises, and the calls can
    be captured into a CUDA graph.  status holds DITANGO_ERR_BOUNDS after a
    request that did not fit or a page number out of range.  The buffers are
    one batch's: calls that may overlap on the GPU need objects of their own.
    data and block_table may be given (a cache that already exists).

    The layers of a model have pages of their own and one batch: `like`, an
    object of the same sizes, lends its tables, lengths, slots, status, and
    scratch, so that tables() is called once, on any of them.  Their calls must
    follow one another (one stream).

    tables() takes pages from free_pages[0] on, in a replayed graph too.  Before
    the next step the taken ones go to the end, without a look at pages_used:

        n = torch.arange(len(free), device=free.device)     # kept
        free.copy_(free[(n + cache.pages_used) % len(free)])
    """

    def __init__(self, n_pages, Hkv, d, max_requests, max_blocks, max_tokens, H=None, device="cuda",
                 data=None, block_table=None, like=None):
        import torch
        for name, v in (("n_pages", n_pages), ("Hkv", Hkv), ("max_requests", max_requests),
                        ("max_blocks", max_blocks), ("max_tokens", max_tokens)):
            if int(v) < 1:
                raise ValueError(f"{name} must be >= 1")
        if d not in (64, 96, 128):
            raise ValueError(f"head dimension {d}: 64, 96 or 128 is required")
        H = Hkv if H is None else H
        if H < 1 or H % Hkv:
            raise ValueError(f"{H} query heads are not a multiple of {Hkv} key heads")
        if like is not None:
            if not isinstance(like, KV4Cache):
                raise TypeError(f"like: a KV4Cache is required, got {type(like).__name__}")
            sizes = (Hkv, H, d, max_requests, max_blocks, max_tokens)
            if sizes != (like.Hkv, like.H, like.d, like.max_requests, like.max_blocks, like.max_tokens):
                raise ValueError("like: an object of the same heads, dimension, requests, blocks and tokens")
            if n_pages < like.n_pages:
                raise ValueError(f"{n_pages} pages, the tables of `like` hold numbers up to {like.n_pages}")
            if block_table is not None:
                raise ValueError("like and block_table exclude each other")
            block_table = like.block_table
            device = like.device
        dev = torch.device(device if data is None else data.device)
        if like is not None and dev != like.device:
            raise ValueError(f"data: on {dev}, the buffers of `like` are on {like.device}")
        if dev.type != "cuda":
            raise ValueError(f"the history lives on a CUDA device, not {dev}")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.n_pages, self.Hkv, self.H, self.d = n_pages, Hkv, H, d
        self.max_requests, self.max_blocks, self.max_tokens = max_requests, max_blocks, max_tokens
        # requests of the last tables() call
        self._batch = {"requests": max_requests} if like is None else like._batch
        shape = (n_pages, Hkv, PAGE * (d + 8))
        if data is None:
            data = torch.zeros(shape, dtype=torch.uint8, device=dev)
        else:
            check_tensor(data, "data", shape, (torch.uint8,), contiguous=True)
        self.data = data
        shape = (max_requests, max_blocks)
        if block_table is None:
            block_table = torch.zeros(shape, dtype=torch.int32, device=dev)
        else:
            _need(block_table, "block_table", shape, (torch.int32,), dev, contiguous=True)
        self.block_table = block_table
        self.sum_codes = torch.zeros((n_pages, Hkv, d), dtype=torch.int8, device=dev)
        self.sum_scale = torch.zeros((n_pages, Hkv), dtype=torch.float32, device=dev)
        if like is not None:
            for name in ("kv_len", "q_off", "slot_map", "pages_used", "status", "ws_bytes", "workspace",
                         "_q_codes", "_q_scale", "_lists"):
                setattr(self, name, getattr(like, name))
        else:
            i32 = dict(dtype=torch.int32, device=dev)
            self.kv_len = torch.zeros(max_requests, **i32)
            self.q_off = torch.zeros(max_requests + 1, **i32)
            self.slot_map = torch.full((max_tokens,), -1, dtype=torch.int64, device=dev)
            self.pages_used = torch.zeros(1, **i32)
            self.status = torch.zeros(1, **i32)
            # the attention's partial states and counters (each launch leaves the counters at zero)
            self.ws_bytes = ditango_kv4_attn_workspace_size(d)
            self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=dev)
            # room for the single tokens' 8-bit codes, for select()
            self._q_codes = torch.empty((max_requests, H, d), dtype=torch.int8, device=dev)
            self._q_scale = torch.empty((max_requests, H), dtype=torch.float32, device=dev)
            self._lists = {}
        self.kv = kv4(n_pages, Hkv, d, self.data)
        self._run = _Launcher(dev)
        self._kv = _abi.C.byref(self.kv)

    @property
    def n_requests(self):
        return self._batch["requests"]

    @n_requests.setter
    def n_requests(self, n):
        self._batch["requests"] = n

    def _lengths(self, name, t, n=None):
        import torch
        if not isinstance(t, torch.Tensor) or t.dim() != 1:
            raise TypeError(f"{name}: a one-dimensional tensor is required")
        _need(t, name, t.shape if n is None else (n,), (torch.int32,), self.device, contiguous=True)

    def tables(self, ctx_len, new_len, free_pages, stream=None):
        """Tables of a batch: request r holds ctx_len[r] tokens and gets
        new_len[r] more; missing pages come from free_pages, in order
        (pages_used says how many were taken).  kv_len holds the new lengths:
        pass a copy of it as the next step's ctx_len."""
        self._lengths("ctx_len", ctx_len)
        R = ctx_len.shape[0]
        if not 1 <= R <= self.max_requests:
            raise ValueError(f"{R} requests, the tables hold 1 to {self.max_requests}")
        self._lengths("new_len", new_len, R)
        self._lengths("free_pages", free_pages)
        n_free = free_pages.shape[0]
        self._run("ditango_block_tables", stream, R, self.max_blocks, self.max_tokens, self.n_pages,
                  ctx_len.data_ptr(), new_len.data_ptr(), free_pages.data_ptr() if n_free else None, n_free,
                  self.block_table.data_ptr(), self.kv_len.data_ptr(), self.q_off.data_ptr(),
                  self.slot_map.data_ptr(), self.pages_used.data_ptr(), self.status.data_ptr())
        self.n_requests = R

    def _rows(self, K, V, slots):
        import torch
        T = K.shape[0] if isinstance(K, torch.Tensor) and K.dim() == 3 else -1
        shape, dev = (T, self.Hkv, self.d), self.device
        _need(K, "K", shape, (torch.bfloat16,), dev)
        _need(V, "V", shape, (torch.bfloat16,), dev)
        if slots is None:
            if T > self.max_tokens:
                raise ValueError(f"{T} tokens, the slot map holds {self.max_tokens}")
            slots = self.slot_map
        else:
            _need(slots, "slots", (T,), (torch.int64,), dev, contiguous=True)
        run = self._run
        return T, K.data_ptr(), V.data_ptr(), run.strides(K, 2), run.strides(V, 2), slots.data_ptr()

    def write(self, K, V, slots=None, stream=None):
        """Quantise K, V [T, Hkv, d] into the slots (default: the slot map of
        the last tables() call; -1 leaves a token out)."""
        self._run("ditango_kv4_write", stream, self._kv, *self._rows(K, V, slots), self.status.data_ptr())

    def read(self, slots, K, V, stream=None):
        """Slots back as bf16 rows of K, V [T, Hkv, d] (rows of -1 are left alone)."""
        self._run("ditango_kv4_read", stream, self._kv, *self._rows(K, V, slots), self.status.data_ptr())

    def summarize(self, ctx_len, stream=None):
        """Refresh the summaries of the pages that got tokens behind ctx_len[r]."""
        self._lengths("ctx_len", ctx_len, self.n_requests)
        self._run("ditango_kv4_summary", stream, self._kv, self.n_requests, self.max_blocks,
                  ctx_len.data_ptr(), self.kv_len.data_ptr(), self.block_table.data_ptr(),
                  self.sum_codes.data_ptr(), self.sum_scale.data_ptr(), self.status.data_ptr())

    def select(self, Q, k, band=0, sink=0, stream=None):
        """(sel, count): the k best pages for one query token a request, Q
        [n_requests, H, d]; the last band + 1 pages and the first sink pages
        are always among them.  The lists are this object's: the next call
        overwrites them."""
        import torch
        R, H, d = self.n_requests, self.H, self.d
        _need(Q, "Q", (R, H, d), (torch.bfloat16,), self.device)
        if k < 0 or sink < 0 or band < -1:
            raise ValueError("k and sink must be >= 0, band >= -1")
        room = max(1, k, sink + (1 + 2 * band if band >= 0 else 0))
        if room not in self._lists:          # one pair of buffers a width, for any number of requests
            self._lists[room] = (
                torch.empty((self.max_requests, self.Hkv, room), dtype=torch.int32, device=self.device),
                torch.empty((self.max_requests, self.Hkv), dtype=torch.int32, device=self.device))
        sel, count = self._lists[room]
        if R != self.max_requests:
            sel, count = sel[:R], count[:R]
        run = self._run
        run("ditango_kv4_select", stream, self._kv, R, H, self.max_blocks, k, band, sink, room, Q.data_ptr(),
            run.strides(Q, 2), self.sum_codes.data_ptr(), self.sum_scale.data_ptr(), self.block_table.data_ptr(),
            self.kv_len.data_ptr(), self._q_codes.data_ptr(), self._q_scale.data_ptr(), sel.data_ptr(),
            count.data_ptr(), self.status.data_ptr())
        return sel, count

    def attend(self, Q, out, out_lse=None, max_q=None, causal=False, scale=0.0, sel=None, sel_count=None,
               stream=None):
        """O and lse of the new tokens Q [T, H, d] over their requests' pages
        (with sel, sel_count: over the listed pages).  out is bf16 or float32
        [T, H, d], out_lse float32 [T, H]; both may be strided views, such as a
        slot of a PartitionedAttention's state buffer.  max_q bounds the new
        tokens of one request (default T)."""
        import torch
        T = Q.shape[0] if isinstance(Q, torch.Tensor) and Q.dim() == 3 else -1
        shape = (T, self.H, self.d)
        dev = self.device
        _need(Q, "Q", shape, (torch.bfloat16,), dev)
        _need(out, "out", shape, (torch.bfloat16, torch.float32), dev)
        if out_lse is not None:
            _lse(out_lse, (T, self.H), dev)
        if (sel is None) != (sel_count is None):
            raise ValueError("sel and sel_count go together")
        room = 0
        if sel is not None:
            room = _width(sel)
            _need(sel, "sel", (self.n_requests, self.Hkv, room), (torch.int32,), dev, contiguous=True)
            _need(sel_count, "sel_count", (self.n_requests, self.Hkv), (torch.int32,), dev, contiguous=True)
        run = self._run
        run("ditango_kv4_attn", stream, self._kv, self.n_requests, self.H, T, T if max_q is None else max_q,
            self.max_blocks, Q.data_ptr(), run.strides(Q, 2), self.q_off.data_ptr(), self.kv_len.data_ptr(),
            self.block_table.data_ptr(), _addr(sel), _addr(sel_count), room, scale, 1 if causal else 0,
            out.data_ptr(), 1 if out.dtype == torch.float32 else 0, run.strides(out, 2), _addr(out_lse),
            None if out_lse is None else run.strides(out_lse, 2), self.workspace.data_ptr(), self.ws_bytes,
            self.status.data_ptr())


class BlockSparseAttention:
    """Attention of 128-query blocks over the 64-key blocks each selects.

    Q [B, H, Nq, d], K and V [B, Hkv, Nk, d], bf16 with any (b, h, n) strides.
    The lists hold, per key head and query block, the blocks within band of the
    query block's own ones (band = -1: none), the first sink blocks and the best
    others by the scores of block means, k in all.  select() fills sel and
    sel_count (and q_/k_ summaries, and k_mean, the means of the key blocks);
    attend() takes those or any other lists; step() does both.  The buffers are
    one call's: calls that may overlap on the GPU need objects of their own.
    """

    def __init__(self, B, H, Nq, Nk, d, k, band=0, sink=0, Hkv=None, device="cuda"):
        import torch
        Hkv = H if Hkv is None else Hkv
        for name, v in (("B", B), ("H", H), ("Hkv", Hkv), ("Nq", Nq), ("Nk", Nk)):
            if int(v) < 1:
                raise ValueError(f"{name} must be >= 1")
        if d not in (64, 96, 128):
            raise ValueError(f"head dimension {d}: 64, 96 or 128 is required")
        if H % Hkv:
            raise ValueError(f"{H} query heads are not a multiple of {Hkv} key heads")
        if k < 0 or sink < 0 or band < -1:
            raise ValueError("k and sink must be >= 0, band >= -1")
        dev = torch.device(device)
        if dev.type != "cuda":
            raise ValueError(f"the lists live on a CUDA device, not {dev}")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.B, self.H, self.Hkv, self.Nq, self.Nk, self.d = B, H, Hkv, Nq, Nk, d
        self.k, self.band, self.sink = k, band, sink
        self.n_q, self.n_k = -(-Nq // QBLOCK), -(-Nk // PAGE)
        per = QBLOCK // PAGE
        self.room = max(1, k, sink + (per + 2 * band if band >= 0 else 0))
        f32, i32, i8 = (dict(dtype=t, device=dev) for t in (torch.float32, torch.int32, torch.int8))
        self.q_codes = torch.empty((B, H, self.n_q, d), **i8)
        self.q_scale = torch.empty((B, H, self.n_q), **f32)
        self.k_codes = torch.empty((B, Hkv, self.n_k, d), **i8)
        self.k_scale = torch.empty((B, Hkv, self.n_k), **f32)
        self.k_mean = torch.empty((B, Hkv, self.n_k, d), **f32)
        self.sel = torch.full((B, Hkv, self.n_q, self.room), -1, **i32)
        self.sel_count = torch.zeros((B, Hkv, self.n_q), **i32)
        self.status = torch.zeros(1, **i32)
        self._run = _Launcher(dev)

    def _check_len(self, k_len):
        import torch
        if k_len is not None:
            _need(k_len, "k_len", (self.B,), (torch.int32,), self.device, contiguous=True)

    def select(self, Q, K, k_len=None, stream=None):
        """(sel, sel_count) for Q and K; k_len [B] int32 (device) bounds the
        valid keys of each batch entry."""
        import torch
        B, H, Hkv, d = self.B, self.H, self.Hkv, self.d
        _need(Q, "Q", (B, H, self.Nq, d), (torch.bfloat16,), self.device)
        _need(K, "K", (B, Hkv, self.Nk, d), (torch.bfloat16,), self.device)
        self._check_len(k_len)
        run, length = self._run, _addr(k_len)
        q_codes, q_scale = self.q_codes.data_ptr(), self.q_scale.data_ptr()
        k_codes, k_scale = self.k_codes.data_ptr(), self.k_scale.data_ptr()
        run("ditango_block_summaries", stream, B, H, Hkv, self.Nq, self.Nk, d, Q.data_ptr(), run.strides(Q, 3),
            K.data_ptr(), run.strides(K, 3), length, q_codes, q_scale, k_codes, k_scale, self.k_mean.data_ptr())
        run("ditango_block_select", stream, B, H, Hkv, self.n_q, self.n_k, d, self.k, self.band, self.sink,
            QBLOCK // PAGE, self.room, q_codes, q_scale, k_codes, k_scale, None, 0, length,
            self.sel.data_ptr(), self.sel_count.data_ptr(), self.status.data_ptr())
        return self.sel, self.sel_count

    def attend(self, Q, K, V, out, out_lse=None, sel=None, sel_count=None, k_len=None, scale=0.0,
               stream=None):
        """O (and lse [B, H, Nq]) of every query block over its listed key
        blocks: the object's lists, or sel [B, Hkv, n_q, any] and sel_count.
        out and out_lse may be strided views, such as a slot of a
        PartitionedAttention's state buffer."""
        import torch
        B, H, Hkv, Nq, d = self.B, self.H, self.Hkv, self.Nq, self.d
        dev, bf16 = self.device, (torch.bfloat16,)
        _need(Q, "Q", (B, H, Nq, d), bf16, dev)
        _need(K, "K", (B, Hkv, self.Nk, d), bf16, dev)
        _need(V, "V", (B, Hkv, self.Nk, d), bf16, dev)
        _need(out, "out", (B, H, Nq, d), (torch.float32, torch.bfloat16), dev)
        if out_lse is not None:
            _lse(out_lse, (B, H, Nq), dev)
        if (sel is None) != (sel_count is None):
            raise ValueError("sel and sel_count go together")
        if sel is None:
            sel, sel_count = self.sel, self.sel_count
        else:
            _need(sel, "sel", (B, Hkv, self.n_q, _width(sel)), (torch.int32,), dev, contiguous=True)
            _need(sel_count, "sel_count", (B, Hkv, self.n_q), (torch.int32,), dev, contiguous=True)
        self._check_len(k_len)
        run = self._run
        run("ditango_block_attn_strided", stream, B, H, Hkv, Nq, self.Nk, d, Q.data_ptr(), K.data_ptr(), V.data_ptr(),
            run.strides(Q, 3), run.strides(K, 3), run.strides(V, 3), sel.data_ptr(), sel_count.data_ptr(),
            sel.shape[-1], _addr(k_len), scale, out.data_ptr(), 1 if out.dtype == torch.float32 else 0,
            run.strides(out, 3), _addr(out_lse), None if out_lse is None else run.strides(out_lse, 3),
            self.status.data_ptr())

    def step(self, Q, K, V, out, out_lse=None, k_len=None, scale=0.0, stream=None):
        """select, then attend."""
        self.select(Q, K, k_len, stream)
        self.attend(Q, K, V, out, out_lse, k_len=k_len, scale=scale, stream=stream)
