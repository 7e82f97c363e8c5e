"""A KV cache in pages: the handle that keeps its tensors and makes the paged calls of graft.h.

``PagedCache`` wraps caller-owned pools and tables (nothing is copied) and
checks them once; its methods check what changes from call to call, and
enqueue one library call each on the current stream of the pools' device:

    cache.reserve(new_rows)                 pages for the step's rows (copy on write)
    cache.plan(q_start, N, Hq, max_new)     once a step
    for every layer:
        q = cache.append(l, Q, K, V, q_start, inv_freq=...)   rotary, new rows into their pages
        o = cache.attend(l, q, scale, mask)                   attention over the pages
    cache.compact(path, acc_len)            accepted tree rows kept
    cache.fork(src, dst), cache.free(seqs)  sequences that share pages; pages given back

Layers with a sliding window take a plan of their own, plan(..., window=, first=), and attend(..., window=, first=); a
step's plans stand side by side.

reserve, append, plan and compact take ``active`` ([n_seqs] bool on the device): sequences that are False there take no
part, so a batch keeps its shape (and a captured step its graph) while sequences come and go.

The buffers a handle allocates (plan, workspaces) grow when a call needs
more and are kept as long as the handle lives, so captured graphs stay
valid; a call that would have to grow one while a graph is being captured is
refused: run it once before.  Calls of one handle share these buffers: order
them on one stream or with events, captured graphs of one handle too.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import binding as gb

# the calls behind torch.cuda.current_device and current_stream, without the objects those build (3 us a call)
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream

_Reference = type(ctypes.byref(ctypes.c_int()))

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


def _kind(window: Optional[int], first: int):
    """What tells the plans of a step apart: (window, first), or None without a window."""
    if window is None:
        if first != 0:
            raise ValueError("first needs a window")
        return None
    whole = isinstance(window, int) and isinstance(first, int) and not isinstance(window, bool) and not isinstance(first, bool)
    if not (whole and 1 <= window < 2**31 and 0 <= first < 2**31):
        raise ValueError("window must be at least 1, first at least 0 (32 bits)")
    return window, first


class PagedCache:
    """Paged cache over per-layer pools ``K``, ``V`` ([num_pages][page_rows][Hkv][128] each, bf16 or fp16).

    block_table [n_seqs][max_pages], lengths [n_seqs] int32; held [n_seqs] and page_refs [num_pages] int32 are
    needed by reserve, fork and free alone; with them append and compact write only to pages that a sequence holds
    alone.  ``status`` collects the GRAFT_STATUS_* bits of every call.
    """

    def __init__(self, K: Sequence[torch.Tensor], V: Sequence[torch.Tensor], block_table: torch.Tensor,
                 lengths: torch.Tensor, page_refs: Optional[torch.Tensor] = None,
                 held: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
        K, V = list(K), list(V)
        if not K or len(K) != len(V):
            raise ValueError("K and V must hold one pool per layer")
        if not isinstance(K[0], torch.Tensor) or K[0].dim() != 4:
            raise ValueError("a pool must be a tensor [num_pages][page_rows][Hkv][head_dim]")
        self.dtype = K[0].dtype
        if self.dtype not in _DTYPES:
            raise ValueError(f"pools must be bfloat16 or float16, got {self.dtype}")
        P, R, H, d = K[0].shape
        for name, pools in (("K", K), ("V", V)):
            for i, t in enumerate(pools):
                gb._need(t, f"{name}[{i}]", self.dtype, (P, R, H, d))
                if t.data_ptr() % 16:  # (compact and reserve take the pools from device arrays, which no call can check)
                    raise ValueError(f"{name}[{i}] must be 16-byte aligned")
        self.device = K[0].device
        gb._need(block_table, "block_table", torch.int32)
        if block_table.dim() != 2:
            raise ValueError("block_table must be [n_seqs][max_pages]")
        S, M = block_table.shape
        gb._need(lengths, "lengths", torch.int32, (S,))
        if held is not None:
            gb._need(held, "held", torch.int32, (S,))
        if page_refs is not None:
            gb._need(page_refs, "page_refs", torch.int32, (P,))
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device) if status is None else status
        gb._need(self.status, "status", torch.int32)
        self.K, self.V, self.block_table, self.lengths = K, V, block_table, lengths
        self.page_refs, self.held = page_refs, held
        for name, t in (("block_table", block_table), ("lengths", lengths), ("held", held), ("page_refs", page_refs),
                        ("status", self.status), *((f"K[{i}]", t) for i, t in enumerate(K)),
                        *((f"V[{i}]", t) for i, t in enumerate(V))):
            if t is not None and t.device != self.device:
                raise ValueError(f"{name} must be on {self.device}, the first pool's device")
        self.n_seqs, self.max_pages, self.page_rows, self.num_pages, self.Hkv = S, M, R, P, H
        self._index = self.device.index
        self._k = gb.layer_pointers(K, self.device)
        self._v = gb.layer_pointers(V, self.device)
        self._kp = [t.data_ptr() for t in K]
        self._vp = [t.data_ptr() for t in V]
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.struct = gb.GraftPagedCache(_DTYPES[self.dtype], H, d, R, P, S, M, len(K), ptr(block_table), ptr(lengths),
                                         ptr(held), ptr(page_refs), self._k.data_ptr(), self._v.data_ptr(),
                                         ptr(self.status))
        self._c = ctypes.addressof(self.struct)
        self._lib = gb.lib()
        self._structs = {}      # address of an ``active`` tensor -> the struct with it
        self._plan_of = None    # (N, Hq, max_new, tree) of the last plan
        self._window_plans = {}  # (window, first) -> the same of the last plan with that window
        self._attended = set()   # kinds (None, (window, first)) whose plan has been attended
        self._sizes = {}        # (N, Hq, max_new) -> bytes of plan and workspace
        self._buffers = {}      # name (a windowed plan's: its window and first) -> buffer in use
        self._kept = []         # buffers outgrown: captured graphs may still use them
        # a cache the kernels cannot take is refused here
        n = ctypes.c_size_t()
        gb._check(self._lib.graft_paged_plan_size(self._c, 0, H, 0, ctypes.byref(n)), "PagedCache")

    # ------------------------------------------------------------------ helpers
    def _buffer(self, name: str, nbytes: int, zero: bool) -> torch.Tensor:
        t = self._buffers.get(name)
        if t is None or t.numel() < nbytes:
            with torch.cuda.device(self._index):
                capturing = torch.cuda.is_current_stream_capturing()
            if capturing:
                raise ValueError(f"the {name if isinstance(name, str) else 'plan'} buffer must grow: run the call once before capturing it")
            if t is not None:
                self._kept.append(t)
                nbytes = max(nbytes, 2 * t.numel())
            make = torch.zeros if zero else torch.empty
            t = self._buffers[name] = make(nbytes, dtype=torch.uint8, device=self.device)
        return t

    def _with(self, active):
        """The cache's struct with ``active`` in it (None: without), as the calls take it.  (A struct each, never changed:
        calls of other host threads may be reading theirs.)  What it returned may be given to it again: a step with many
        layers asks once."""
        if active is None:
            return self._c
        if type(active) is _Reference:
            return active
        at = self._need(active, "active", torch.bool, (self.n_seqs,))
        c = self._structs.get(at)
        if c is None:
            c = gb.GraftPagedCache.from_buffer_copy(self.struct)
            c.active = at
            if len(self._structs) < 256:
                self._structs[at] = c
        return ctypes.byref(c)

    def _call(self, name: str, c, *args) -> None:
        stream = _raw_stream(self._index)
        if _current_device() == self._index:
            rc = getattr(self._lib, name)(c, *args, stream)
        else:
            with torch.cuda.device(self._index):
                rc = getattr(self._lib, name)(c, *args, stream)
        if rc:
            gb._check(rc, name)

    # (the checks run once a tensor and call, a dozen times a step and layer: the usual case comes first, and only
    # what it does not take is looked at again for a message)
    def _need(self, t: torch.Tensor, name: str, dtype: torch.dtype, shape) -> int:
        """Checks a dense tensor on the cache's device; returns its address."""
        try:
            if t.dtype is dtype and t.get_device() == self._index and t.shape == shape and t.is_contiguous():
                return t.data_ptr()
        except AttributeError:
            raise TypeError(f"{name} must be a tensor") from None
        gb._need(t, name, dtype, shape)
        raise ValueError(f"{name} must be on {self.device}")

    def _rows(self, t: torch.Tensor, name: str, N: int, H: int):
        """Checks [N][H][128] rows whose heads are contiguous; returns address and row stride."""
        width = H * 128
        try:
            if t.dtype is self.dtype and t.get_device() == self._index and t.shape == (N, H, 128):
                s0, s1, s2 = t.stride()
                if s2 == 1 and s1 == 128 and s0 >= width and not s0 & 7:
                    return t.data_ptr(), s0
        except AttributeError:
            raise TypeError(f"{name} must be a tensor") from None
        if t.dtype is not self.dtype or t.device != self.device:
            raise ValueError(f"{name} must be {self.dtype} on {self.device}")
        if t.shape != (N, H, gb.HEAD_DIM):
            raise ValueError(f"{name} must have shape {(N, H, gb.HEAD_DIM)}, got {tuple(t.shape)}")
        s0, s1, s2 = t.stride()
        if N <= 1 or H == 0:
            s0 = width  # (the stride of a single row, or of no columns, means nothing)
        if H and (s2 != 1 or (H > 1 and s1 != gb.HEAD_DIM)):
            raise ValueError(f"{name} must have contiguous heads")
        if s0 < width or s0 % 8:
            raise ValueError(f"{name}'s rows must be at least {width} elements apart, by a multiple of 8")
        return t.data_ptr(), s0

    def _layer(self, layer: int) -> int:
        if not 0 <= layer < len(self._kp):
            raise ValueError(f"layer must be in [0, {len(self._kp)})")
        return layer

    # ------------------------------------------------------------------ calls
    def append(self, layer: int, Q, K, V, q_start, inv_freq=None, interleaved: bool = False, positions=None,
               factor: float = 1.0, out=None, active=None, q_norm=None, k_norm=None, eps: float = 1e-6):
        """graft_rope_append: rotates Q and K ([N][H][128], rows may be strided), writes K and V to their pages.

        Returns the rotated Q (``out``, which may be Q itself).  Q may be None.  Without inv_freq nothing is rotated.
        ``q_norm`` and ``k_norm`` ([128] float32 weights, either may be None) norm the heads of Q and K first
        (graft_norm_rope_append)."""
        layer = self._layer(layer)
        if not isinstance(K, torch.Tensor) or K.dim() != 3:
            raise ValueError("K must be [N][Hkv][128]")
        N = K.shape[0]
        kp, ks = self._rows(K, "K", N, self.Hkv)
        vp, vs = self._rows(V, "V", N, self.Hkv)
        qp = op = None
        qs = os = Hq = 0
        if Q is not None:
            if not isinstance(Q, torch.Tensor) or Q.dim() != 3:
                raise ValueError("Q must be [N][Hq][128]")
            Hq = Q.shape[1]
            qp, qs = self._rows(Q, "Q", N, Hq)
            if out is None:
                out = torch.empty((N, Hq, gb.HEAD_DIM), dtype=self.dtype, device=self.device)
            op, os = self._rows(out, "out", N, Hq)
        starts = self._need(q_start, "q_start", torch.int32, (self.n_seqs + 1,))
        pos = None if positions is None else self._need(positions, "positions", torch.int32, (N,))
        fp, rot = None, 0
        if inv_freq is not None:
            rot = 2 * inv_freq.numel()
            fp = self._need(inv_freq, "inv_freq", torch.float64, (rot // 2,))
        head = (self._kp[layer], self._vp[layer], N, Hq, starts, pos, fp, rot, 1 if interleaved else 0, float(factor))
        if q_norm is None and k_norm is None:
            self._call("graft_rope_append", self._with(active), *head, qp, qs, kp, ks, vp, vs, op, os)
        else:
            d = (gb.HEAD_DIM,)
            qw = None if q_norm is None else self._need(q_norm, "q_norm", torch.float32, d)
            kw = None if k_norm is None else self._need(k_norm, "k_norm", torch.float32, d)
            self._call("graft_norm_rope_append", self._with(active), *head, qw, kw, float(eps), qp, qs, kp, ks, vp, vs,
                       op, os)
        return out

    def plan(self, q_start, N: int, Hq: int, max_new: int, tree: bool = False, active=None, window: Optional[int] = None,
             first: int = 0) -> None:
        """graft_paged_plan for a step of N rows; serves every attend() until the next step's plan().

        With ``window`` (and ``first``) graft_paged_plan_window, for the attend()s with the same two: a step whose
        layers are of several kinds makes a plan of each.  A kind that is planned again begins the next step: plans of
        other kinds that have been attended are dropped, so that each is planned anew before it is attended.  (A handle
        keeps a plan buffer for every kind it has seen.)"""
        kind = _kind(window, first)
        again = self._drop(kind)  # (a plan that is refused leaves none)
        starts = self._need(q_start, "q_start", torch.int32, (self.n_seqs + 1,))
        key = (N, Hq, max_new)
        sizes = self._sizes.get(key)
        if sizes is None:
            a, b = ctypes.c_size_t(), ctypes.c_size_t()
            with torch.cuda.device(self._index):
                gb._check(self._lib.graft_paged_plan_size(self._c, *key, ctypes.byref(a)), "graft_paged_plan_size")
                gb._check(self._lib.graft_paged_attention_workspace_size(self._c, *key, ctypes.byref(b)),
                          "graft_paged_attention_workspace_size")
            if len(self._sizes) >= 4096:
                self._sizes.clear()
            sizes = self._sizes[key] = (a.value, b.value)
        buf = self._buffer("plan" if kind is None else kind, sizes[0], False)
        self._buffer("attention", sizes[1], True)
        if kind is None:
            self._call("graft_paged_plan", self._with(active), N, Hq, starts, max_new, 1 if tree else 0, buf.data_ptr(),
                       buf.numel())
        else:
            self._call("graft_paged_plan_window", self._with(active), N, Hq, starts, max_new, 1 if tree else 0, *kind,
                       buf.data_ptr(), buf.numel())
        if again:
            for other in list(self._attended):
                self._drop(other)
        if kind is None:
            self._plan_of = (N, Hq, max_new, bool(tree))
        else:
            self._window_plans[kind] = (N, Hq, max_new, bool(tree))

    def _drop(self, kind) -> bool:
        """Forgets the plan of a kind; whether there was one."""
        self._attended.discard(kind)
        if kind is not None:
            return self._window_plans.pop(kind, None) is not None
        there, self._plan_of = self._plan_of is not None, None
        return there

    def attend(self, layer: int, Q, scale: float, mask=None, out=None, tuning=None, window: Optional[int] = None,
               first: int = 0):
        """graft_paged_attention of the planned step: Q [N][Hq][128] (rows may be strided), mask [N] int64 (the
        ancestor bits) for a tree plan; returns O [N][Hq][128].  ``tuning`` (a GraftAttnTuning or a dict of its
        fields, of which wait_ns alone may be set) selects graft_paged_attention_ex.  With ``window`` (and ``first``)
        graft_paged_attention_window: a row sees the last ``window`` positions and the ``first`` tokens alone."""
        kind = _kind(window, first)
        plan_of = self._plan_of if kind is None else self._window_plans.get(kind)
        if plan_of is None:
            raise ValueError("attend() needs a plan() of the step" + ("" if kind is None else " with this window"))
        N, Hq, max_new, tree = plan_of
        if tree != (mask is not None):
            raise ValueError("a plan with tree=True takes a mask, one without takes none")
        layer = self._layer(layer)
        qp, qs = self._rows(Q, "Q", N, Hq)
        if out is None:
            out = torch.empty((N, Hq, gb.HEAD_DIM), dtype=self.dtype, device=self.device)
        op = self._need(out, "out", self.dtype, (N, Hq, gb.HEAD_DIM))
        mp = None if mask is None else self._need(mask, "mask", torch.int64, (N,))
        plan, ws = self._buffers["plan" if kind is None else kind], self._buffers["attention"]
        if kind is not None:
            tuning = gb._tuning(tuning)
            self._call("graft_paged_attention_window", self._c, self._kp[layer], self._vp[layer], N, Hq, max_new, *kind,
                       plan.data_ptr(), plan.numel(), qp, qs, mp, float(scale), op,
                       None if tuning is None else ctypes.addressof(tuning), ws.data_ptr(), ws.numel())
        elif tuning is None:
            self._call("graft_paged_attention", self._c, self._kp[layer], self._vp[layer], N, Hq, max_new,
                       plan.data_ptr(), plan.numel(), qp, qs, mp, float(scale), op, ws.data_ptr(), ws.numel())
        else:
            tuning = gb._tuning(tuning)
            self._call("graft_paged_attention_ex", self._c, self._kp[layer], self._vp[layer], N, Hq, max_new,
                       plan.data_ptr(), plan.numel(), qp, qs, mp, float(scale), op, ctypes.addressof(tuning),
                       ws.data_ptr(), ws.numel())
        self._attended.add(kind)
        return out

    def compact(self, path, acc_len, lengths_out=None, active=None):
        """graft_pages_compact: path [n_seqs][Kmax], acc_len [n_seqs]; lengths advance in place unless
        ``lengths_out`` receives them."""
        if not isinstance(path, torch.Tensor) or path.dim() != 2:
            raise ValueError("path must be [n_seqs][Kmax]")
        Kmax = path.shape[1]
        pp = self._need(path, "path", torch.int32, (self.n_seqs, Kmax))
        ap = self._need(acc_len, "acc_len", torch.int32, (self.n_seqs,))
        if lengths_out is None:
            lengths_out = self.lengths
        lp = self._need(lengths_out, "lengths_out", torch.int32, (self.n_seqs,))
        self._call("graft_pages_compact", self._with(active), Kmax, pp, ap, lp)
        return lengths_out

    def _tables(self) -> None:
        if self.held is None or self.page_refs is None:
            raise ValueError("reserve, fork and free need held and page_refs")

    def reserve(self, new_rows, active=None) -> None:
        """graft_pages_reserve: pages for new_rows [n_seqs] more rows of every sequence."""
        self._tables()
        np = self._need(new_rows, "new_rows", torch.int32, (self.n_seqs,))
        ws = self._buffers.get("reserve")
        if ws is None:
            n = ctypes.c_size_t()
            gb._check(self._lib.graft_pages_reserve_workspace_size(self._c, ctypes.byref(n)),
                      "graft_pages_reserve_workspace_size")
            ws = self._buffer("reserve", n.value, False)
        self._call("graft_pages_reserve", self._with(active), np, ws.data_ptr(), ws.numel())

    def fork(self, src, dst) -> None:
        """graft_pages_fork: sequence dst[i] shares the pages of src[i] ([n] int32 each)."""
        self._tables()
        n = src.numel()
        sp = self._need(src, "src", torch.int32, (n,))
        dp = self._need(dst, "dst", torch.int32, (n,))
        self._call("graft_pages_fork", self._c, n, sp, dp)

    def free(self, seqs) -> None:
        """graft_pages_free: gives back the pages of sequences seqs [n] int32."""
        self._tables()
        n = seqs.numel()
        self._call("graft_pages_free", self._c, n, self._need(seqs, "seqs", torch.int32, (n,)))
