"""The paged E4M3 cache: Python binding of the kvs_paged_* calls of include/kvs.h.

Every length, block table and slot is a CUDA tensor of the caller's; no method reads one
on the host, so a step (plan, then append and attend per layer) can be captured in a
graph and replayed while the batch changes.
"""

import collections
import ctypes

import torch

from . import _abi, KVSError, _need, _ptr, _TORCH_DT, lib

PagedPlan = collections.namedtuple("PagedPlan", "row_start kv_len slots positions denied")
PagedPlan.__doc__ = """What one plan made: row_start [n + 1], kv_len [n], slots and positions
[row_capacity], denied [1], all int32 CUDA tensors."""
# the packed rows' starts are also where each request's queries start
PagedPlan.q_start = property(lambda self: self.row_start)


def paged_config_init(**fields):
    """A kvs_paged_config with the library defaults, then the given fields."""
    cfg = _abi.PagedConfig()
    lib().kvs_paged_config_init(ctypes.byref(cfg))
    for k, v in fields.items():
        setattr(cfg, k, v)
    return cfg


def validate_paged_config(cfg):
    """(status, message) of the host-side config check."""
    buf = ctypes.create_string_buffer(512)
    st = lib().kvs_paged_validate_config(ctypes.byref(cfg), buf, len(buf))
    return st, buf.value.decode()


def paged_workspace_bytes(cfg):
    return int(lib().kvs_paged_workspace_bytes(ctypes.byref(cfg)))


class PagedCache:
    """A kvs_paged context bound to a workspace this object owns (a torch uint8 tensor).

    Work goes on `stream`, by default the current stream of the cache's device.  Outputs
    that a method allocates are safe to use on that stream."""

    def __init__(self, cfg, device=None, stream=None):
        st, msg = validate_paged_config(cfg)
        if st != _abi.OK:
            raise KVSError(st, msg)
        self.cfg = _abi.PagedConfig.from_buffer_copy(cfg)
        device = torch.device("cuda" if device is None else device)
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device = device
        nbytes = paged_workspace_bytes(cfg)
        self._ctx = ctypes.c_void_p()
        with torch.cuda.device(device):
            self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
            st = lib().kvs_paged_create(ctypes.byref(cfg), _ptr(self.workspace), nbytes, self._stream(stream)[0],
                                        ctypes.byref(self._ctx))
        if st != _abi.OK:
            raise KVSError(st, "kvs_paged_create failed")
        self.in_dtype = _TORCH_DT[cfg.in_dtype]

    def __del__(self):
        if getattr(self, "_ctx", None) and self._ctx.value:
            try:
                lib().kvs_paged_destroy(self._ctx)
            except Exception:
                pass
            self._ctx = None

    def _check(self, st):
        if st != _abi.OK:
            raise KVSError(st, self.last_error())

    def _stream(self, stream):
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        return ctypes.c_void_p(s.cuda_stream), s

    def _need(self, t, name, dtype, shape):
        _need(t, name, dtype, shape)
        if t.device != self.device:
            raise ValueError("%s must be on %s, got %s" % (name, self.device, t.device))

    def _empty(self, shape, dtype, stream):
        t = torch.empty(shape, dtype=dtype, device=self.device)
        if stream is not None:
            t.record_stream(stream)      # freed memory is not reused before the launch has run
        return t

    def _table(self, block_table, n):
        if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
            raise TypeError("block_table must be a 2-d CUDA tensor")
        self._need(block_table, "block_table", torch.int32, (n, block_table.shape[1]))
        return int(block_table.shape[1])

    def _lengths(self, t, name):
        if not isinstance(t, torch.Tensor) or t.dim() != 1:
            raise TypeError("%s must be a 1-d CUDA tensor" % name)
        self._need(t, name, torch.int32, (t.shape[0],))
        return int(t.shape[0])

    # ---- tables
    def plan(self, ctx_len, new_len, block_table, free_pages, free_count, row_capacity, free_count_out=None,
             kv_len_out=None, stream=None):
        """Pages, slots and positions for new_len[r] tokens behind ctx_len[r] cached ones.
        Fills block_table [n, stride] in place; pages come from the stack free_pages
        [capacity] whose size is free_count [1].  free_count_out (default: free_count)
        and kv_len_out (may be ctx_len) receive the updated state.  Returns a PagedPlan."""
        n = self._lengths(ctx_len, "ctx_len")
        self._need(new_len, "new_len", torch.int32, (n,))
        stride = self._table(block_table, n)
        cap = self._lengths(free_pages, "free_pages")
        self._need(free_count, "free_count", torch.int32, (1,))
        if free_count_out is None:
            free_count_out = free_count
        self._need(free_count_out, "free_count_out", torch.int32, (1,))
        rows = int(row_capacity)
        if rows < 0:
            raise ValueError("row_capacity must be >= 0")
        # one allocation for the small outputs; each part on a 16-byte boundary
        up = lambda x: (x + 3) & ~3  # noqa: E731
        sizes = [n + 1, 0 if kv_len_out is not None else n, rows, rows, 1]
        buf = self._empty((sum(up(x) for x in sizes),), torch.int32, stream)
        parts, at = [], 0
        for x in sizes:
            parts.append(buf[at:at + x])
            at += up(x)
        if kv_len_out is not None:
            self._need(kv_len_out, "kv_len_out", torch.int32, (n,))
            parts[1] = kv_len_out
        p = PagedPlan(*parts)
        self._check(lib().kvs_paged_plan(
            self._ctx, n, _ptr(ctx_len), _ptr(new_len), _ptr(block_table), stride, _ptr(free_pages), cap,
            _ptr(free_count), _ptr(free_count_out), _ptr(p.row_start), _ptr(p.kv_len), _ptr(p.slots),
            _ptr(p.positions), rows, _ptr(p.denied), self._stream(stream)[0]))
        return p

    def slot_map(self, length, block_table, row_capacity, first=None, stream=None):
        """Slots and positions of positions first[r] .. first[r] + length[r] - 1 (first: 0)
        from filled tables.  Returns (row_start [n + 1], slots, positions [row_capacity])."""
        n = self._lengths(length, "length")
        if first is not None:
            self._need(first, "first", torch.int32, (n,))
        stride = self._table(block_table, n)
        rows = int(row_capacity)
        if rows < 0:
            raise ValueError("row_capacity must be >= 0")
        row_start = self._empty((n + 1,), torch.int32, stream)
        slots = self._empty((rows,), torch.int32, stream)
        positions = self._empty((rows,), torch.int32, stream)
        self._check(lib().kvs_paged_slot_map(
            self._ctx, n, None if first is None else _ptr(first), _ptr(length), _ptr(block_table), stride,
            _ptr(row_start), _ptr(slots), _ptr(positions), rows, self._stream(stream)[0]))
        return row_start, slots, positions

    def release(self, kv_len, block_table, free_pages, free_count, stream=None):
        """Return the pages of finished requests (rows of block_table) to the stack."""
        n = self._lengths(kv_len, "kv_len")
        stride = self._table(block_table, n)
        cap = self._lengths(free_pages, "free_pages")
        self._need(free_count, "free_count", torch.int32, (1,))
        self._check(lib().kvs_paged_release(self._ctx, n, _ptr(kv_len), _ptr(block_table), stride, _ptr(free_pages),
                                            cap, _ptr(free_count), self._stream(stream)[0]))

    # ---- tokens
    def _rows(self, slots):
        return self._lengths(slots, "slots"), (self.cfg.num_kv_heads, self.cfg.head_dim)

    def append(self, layer, k, v, slots, stream=None):
        """Store k, v [rows, Hkv, D] (input dtype) at slots [rows]."""
        n, shape = self._rows(slots)
        self._need(k, "k", self.in_dtype, (n,) + shape)
        self._need(v, "v", self.in_dtype, (n,) + shape)
        self._check(lib().kvs_paged_append(self._ctx, layer, n, _ptr(slots), _ptr(k), _ptr(v), self._stream(stream)[0]))

    def gather(self, layer, slots, k_out=None, v_out=None, stream=None):
        """The values at slots [rows]: (k, v), each [rows, Hkv, D] in the input dtype."""
        n, shape = self._rows(slots)
        if k_out is None:
            k_out = self._empty((n,) + shape, self.in_dtype, stream)
        if v_out is None:
            v_out = self._empty((n,) + shape, self.in_dtype, stream)
        self._need(k_out, "k_out", self.in_dtype, (n,) + shape)
        self._need(v_out, "v_out", self.in_dtype, (n,) + shape)
        self._check(lib().kvs_paged_gather(self._ctx, layer, n, _ptr(slots), _ptr(k_out), _ptr(v_out),
                                           self._stream(stream)[0]))
        return k_out, v_out

    def attend_scratch_bytes(self, n_reqs, table_stride, total_q, max_q_len=1, block_mass=False):
        return int(lib().kvs_paged_attend_scratch_bytes(self._ctx, n_reqs, table_stride, total_q, max_q_len,
                                                        int(bool(block_mass))))

    def attend(self, layer, q, block_table, kv_len, q_start=None, max_q_len=1, window=0, block_mass=None, out=None,
               scratch=None, stream=None):
        """Attend q [rows, Hq, D] (input dtype) over the pages; returns out of q's shape and
        type.  Without q_start there is one row per request; with it (int32 [n + 1], a
        plan's row_start) request r's rows are q_start[r] .. q_start[r + 1] - 1, its last
        tokens, at most max_q_len of them.  window > 0: only the last `window` positions.
        block_mass: optional float32 [n, stride] that receives each visible block's mass
        (single-token rows only).  scratch: optional uint8 tensor of attend_scratch_bytes."""
        n = self._lengths(kv_len, "kv_len")
        stride = self._table(block_table, n)
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise TypeError("q must be a 3-d CUDA tensor")
        rows = int(q.shape[0])
        shape = (rows, self.cfg.num_q_heads, self.cfg.head_dim)
        self._need(q, "q", self.in_dtype, shape)
        if q_start is not None:
            self._need(q_start, "q_start", torch.int32, (n + 1,))
        if block_mass is not None:
            self._need(block_mass, "block_mass", torch.float32, (n, stride))
        if out is None:
            out = self._empty(shape, self.in_dtype, stream)
        self._need(out, "out", self.in_dtype, shape)
        if scratch is None:
            scratch = self._empty((self.attend_scratch_bytes(n, stride, rows, max_q_len, block_mass is not None),),
                                  torch.uint8, stream)
        if not scratch.is_cuda or scratch.device != self.device or scratch.dtype != torch.uint8 or not scratch.is_contiguous():
            raise TypeError("scratch must be a contiguous uint8 tensor on %s" % self.device)
        self._check(lib().kvs_paged_attend(
            self._ctx, layer, n, _ptr(block_table), stride, _ptr(kv_len), None if q_start is None else _ptr(q_start),
            rows, max_q_len, window, _ptr(q), _ptr(out), None if block_mass is None else _ptr(block_mass),
            _ptr(scratch), scratch.numel(), self._stream(stream)[0]))
        return out

    # ---- inspection
    def get_status(self, stream=None):
        """Synchronise and return the device status code (0 = OK)."""
        return lib().kvs_paged_get_status(self._ctx, self._stream(stream)[0])

    def clear_error(self, stream=None):
        self._check(lib().kvs_paged_clear_error(self._ctx, self._stream(stream)[0]))

    def last_error(self):
        return lib().kvs_paged_last_error(self._ctx).decode()
