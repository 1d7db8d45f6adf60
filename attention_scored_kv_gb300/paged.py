"""The paged E4M3 cache: Python binding of the kvs_paged_* calls of include/kvs.h.

Every length, block table and slot is a CUDA tensor of the caller's; no method reads one
on the host, so a step (plan, then append and attend per layer) can be captured in a
graph and replayed while the batch changes.
"""

import collections
import ctypes
import importlib.machinery
import importlib.util
import os
import warnings

import torch

from . import _abi, KVSError, _need, _TORCH_DT, lib

_Tensor, _i32, _f32 = torch.Tensor, torch.int32, torch.float32
_empty = torch.empty
# absent where torch is built without CUDA: the host-side calls work there too
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

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
        setattr(cfg, k, _abi.int32(v) if isinstance(getattr(cfg, k, None), int) else v)
    return cfg


def validate_paged_config(cfg):
    """(status, message) of the host-side config check."""
    buf = ctypes.create_string_buffer(512)
    st = lib().kvs_paged_validate_config(ctypes.byref(cfg), buf, len(buf))
    return st, buf.value.decode()


def paged_workspace_bytes(cfg):
    return int(lib().kvs_paged_workspace_bytes(ctypes.byref(cfg)))


_call = None


def _load_call():
    """The extension that makes the calls of a decode step (csrc/paged_call.cpp), bound to the loaded library.
    None where it was not built, or not for this torch: every call then goes through ctypes."""
    global _call
    if _call is None:
        path = os.path.join(os.path.dirname(_abi.LIB_PATH), "_paged_call.so")
        if not os.path.exists(path):
            warnings.warn("_paged_call.so is not built (%s): paged calls take 5 to 20 us longer each" % path)
            return None
        loader = importlib.machinery.ExtensionFileLoader("_paged_call", path)
        try:
            module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_paged_call", loader))
            loader.exec_module(module)
        except ImportError as e:
            warnings.warn("_paged_call.so does not load (%s): paged calls take 5 to 20 us longer each" % e)
            return None
        module.bind(*(ctypes.cast(getattr(lib(), "kvs_paged_" + f), ctypes.c_void_p).value
                      for f in ("plan", "append", "gather", "attend", "attend_scratch_bytes")))
        _call = module
    return _call


class PagedCache:
    """A kvs_paged context bound to a workspace this object owns (a torch uint8 tensor).

    Work goes on `stream`, by default the current stream of the cache's device.  What a
    method allocates is allocated on that stream, so that no earlier work of another stream
    still uses the memory, and may be used on it and, once that waits for it, on the current
    one.  The workspace outlives the work that any stream has with it; a graph that was
    captured over a cache needs the cache to live as long.

    plan, append, gather and attend on the current stream, with outputs of their own, are
    taken by an extension module, where it is built; it declines what it does not find in
    order, and the method's own checks say why."""

    _fast = None

    def __init__(self, cfg, device=None, stream=None):
        st, msg = validate_paged_config(cfg)
        if st != _abi.OK:
            raise KVSError(st, msg)
        self.cfg = _abi.PagedConfig.from_buffer_copy(cfg)
        device = torch.device("cuda" if device is None else device)
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device, self._index, self._lib = device, device.index, lib()
        nbytes = paged_workspace_bytes(cfg)
        self._ctx = ctypes.c_void_p()
        self._streams = set()                # raw handles of the streams that have used the workspace
        with torch.cuda.device(device):
            with torch.cuda.stream(stream):  # None: the current one
                self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
            st = self._lib.kvs_paged_create(ctypes.byref(cfg), self.workspace.data_ptr(), nbytes, self._stream(stream),
                                            ctypes.byref(self._ctx))
        if st != _abi.OK:
            raise KVSError(st, "kvs_paged_create failed")
        self.in_dtype = _TORCH_DT[cfg.in_dtype]
        self._row = (int(cfg.num_kv_heads), int(cfg.head_dim))
        self._qrow = (int(cfg.num_q_heads), int(cfg.head_dim))
        self._fast = _load_call()
        self._key = (self._ctx.value, self._index, self._row[0], self._qrow[0], self._row[1], cfg.in_dtype == _abi.BF16)

    def __del__(self):
        if getattr(self, "_ctx", None) and self._ctx.value:
            try:
                self._lib.kvs_paged_destroy(self._ctx)
            except Exception:
                pass
            self._ctx = None

    def _check(self, st):
        if st != _abi.OK:
            raise KVSError(st, self.last_error())

    def _stream(self, stream):
        if stream is None:
            raw = _raw_stream(self._index)
        else:
            if stream.device != self.device:
                raise ValueError("stream must be on %s, got one on %s" % (self.device, stream.device))
            raw = stream.cuda_stream
        if raw not in self._streams:
            self._mark(raw, stream)
        return raw

    def _mark(self, raw, stream=None):
        """The workspace's memory is not reused before this stream is done with it."""
        self.workspace.record_stream(torch.cuda.current_stream(self.device) if stream is None else stream)
        self._streams.add(raw)

    # A call of a decode step runs on the GPU for a few microseconds, so the checks are spelled out for the
    # tensors that pass and leave the message to _need.
    def _need(self, t, name, dtype, shape):
        if (t.__class__ is not _Tensor or t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
                or t.get_device() != self._index):
            _need(t, name, dtype, shape)
            if t.device != self.device:
                raise ValueError("%s must be on %s, got %s" % (name, self.device, t.device))
        return t.data_ptr()

    def _need_dims(self, t, name, dtype, dims):
        """As _need for a tensor whose shape is free: its shape."""
        if not isinstance(t, _Tensor) or t.dim() != dims:
            raise TypeError("%s must be a %d-d CUDA tensor" % (name, dims))
        shape = t.shape
        self._need(t, name, dtype, shape)
        return shape

    def _empty(self, shape, dtype, stream):
        if stream is None:
            return _empty(shape, dtype=dtype, device=self.device)
        if stream.device != self.device:
            raise ValueError("stream must be on %s, got one on %s" % (self.device, stream.device))
        with torch.cuda.stream(stream):
            t = _empty(shape, dtype=dtype, device=self.device)
        t.record_stream(torch.cuda.current_stream(self.device))      # where the caller is likely to read it
        return t

    # ---- tables
    def plan(self, ctx_len, new_len, block_table, free_pages, free_count, row_capacity, free_count_out=None,
             kv_len_out=None, stream=None):
        """Pages, slots and positions for new_len[r] tokens behind ctx_len[r] cached ones.
        Fills block_table [n, stride] in place; pages come from the stack free_pages
        [capacity] whose size is free_count [1].  free_count_out (default: free_count)
        and kv_len_out (may be ctx_len) receive the updated state.  Returns a PagedPlan."""
        if stream is None and kv_len_out is None and self._fast is not None:
            if _raw_stream(self._index) not in self._streams:
                self._mark(_raw_stream(self._index))
            r = self._fast.plan(self._key, ctx_len, new_len, block_table, free_pages, free_count,
                                free_count if free_count_out is None else free_count_out, row_capacity)
            if r.__class__ is tuple:
                return PagedPlan(*r)
            if r is not None:
                self._check(r)
        n, = self._need_dims(ctx_len, "ctx_len", _i32, 1)
        stride = self._need_dims(block_table, "block_table", _i32, 2)[1]
        cap, = self._need_dims(free_pages, "free_pages", _i32, 1)
        new = self._need(new_len, "new_len", _i32, (n,))
        table = self._need(block_table, "block_table", _i32, (n, stride))
        count = self._need(free_count, "free_count", _i32, (1,))
        count_out = count if free_count_out is None else self._need(free_count_out, "free_count_out", _i32, (1,))
        rows = int(row_capacity)
        if rows < 0:
            raise ValueError("row_capacity must be >= 0")
        # one allocation for the outputs, slots and positions on 16-byte boundaries
        pad = -rows & 3
        sizes = (rows, pad, rows, n + 1, n, 1)
        out = self._empty((2 * rows + pad + 2 * n + 2,), _i32, stream)
        slots, _, positions, row_start, kv_len, denied = out.split_with_sizes(sizes)
        if kv_len_out is not None:
            self._need(kv_len_out, "kv_len_out", _i32, (n,))
            kv_len = kv_len_out
        at = out.data_ptr()
        start = at + 4 * (2 * rows + pad)
        st = self._lib.kvs_paged_plan(
            self._ctx, n, ctx_len.data_ptr(), new, table, stride, free_pages.data_ptr(), cap, count, count_out,
            start, kv_len.data_ptr(), at, at + 4 * (rows + pad), rows, start + 4 * (2 * n + 1), self._stream(stream))
        if st:
            self._check(st)
        return PagedPlan(row_start, kv_len, slots, positions, denied)

    def slot_map(self, length, block_table, row_capacity, first=None, stream=None):
        """Slots and positions of positions first[r] .. first[r] + length[r] - 1 (first: 0)
        from filled tables.  Returns (row_start [n + 1], slots, positions [row_capacity])."""
        n, = self._need_dims(length, "length", _i32, 1)
        stride = self._need_dims(block_table, "block_table", _i32, 2)[1]
        table = self._need(block_table, "block_table", _i32, (n, stride))
        rows = int(row_capacity)
        if rows < 0:
            raise ValueError("row_capacity must be >= 0")
        row_start = self._empty((n + 1,), _i32, stream)
        slots = self._empty((rows,), _i32, stream)
        positions = self._empty((rows,), _i32, stream)
        self._check(self._lib.kvs_paged_slot_map(
            self._ctx, n, None if first is None else self._need(first, "first", _i32, (n,)), length.data_ptr(), table,
            stride, row_start.data_ptr(), slots.data_ptr(), positions.data_ptr(), rows, self._stream(stream)))
        return row_start, slots, positions

    def release(self, kv_len, block_table, free_pages, free_count, stream=None):
        """Return the pages of finished requests (rows of block_table) to the stack."""
        n, = self._need_dims(kv_len, "kv_len", _i32, 1)
        stride = self._need_dims(block_table, "block_table", _i32, 2)[1]
        cap, = self._need_dims(free_pages, "free_pages", _i32, 1)
        self._check(self._lib.kvs_paged_release(
            self._ctx, n, kv_len.data_ptr(), self._need(block_table, "block_table", _i32, (n, stride)), stride,
            free_pages.data_ptr(), cap, self._need(free_count, "free_count", _i32, (1,)), self._stream(stream)))

    # ---- tokens
    def append(self, layer, k, v, slots, stream=None):
        """Store k, v [rows, Hkv, D] (input dtype) at slots [rows]."""
        if stream is None and self._fast is not None:
            if _raw_stream(self._index) not in self._streams:
                self._mark(_raw_stream(self._index))
            st = self._fast.append(self._key, layer, k, v, slots)
            if st == 0:
                return
            if st is not None:
                self._check(st)
        n, = self._need_dims(slots, "slots", _i32, 1)
        shape = (n,) + self._row
        st = self._lib.kvs_paged_append(
            self._ctx, layer, n, slots.data_ptr(), self._need(k, "k", self.in_dtype, shape),
            self._need(v, "v", self.in_dtype, shape), self._stream(stream))
        if st:
            self._check(st)

    def gather(self, layer, slots, k_out=None, v_out=None, stream=None):
        """The values at slots [rows]: (k, v), each [rows, Hkv, D] in the input dtype."""
        if stream is None and k_out is None and v_out is None and self._fast is not None:
            if _raw_stream(self._index) not in self._streams:
                self._mark(_raw_stream(self._index))
            r = self._fast.gather(self._key, layer, slots)
            if r.__class__ is tuple:
                return r
            if r is not None:
                self._check(r)
        n, = self._need_dims(slots, "slots", _i32, 1)
        shape = (n,) + self._row
        if k_out is None:
            k_out = self._empty(shape, self.in_dtype, stream)
        if v_out is None:
            v_out = self._empty(shape, self.in_dtype, stream)
        st = self._lib.kvs_paged_gather(
            self._ctx, layer, n, slots.data_ptr(), self._need(k_out, "k_out", self.in_dtype, shape),
            self._need(v_out, "v_out", self.in_dtype, shape), self._stream(stream))
        if st:
            self._check(st)
        return k_out, v_out

    def attend_scratch_bytes(self, n_reqs, table_stride, total_q, max_q_len=1, block_mass=False):
        return self._lib.kvs_paged_attend_scratch_bytes(self._ctx, n_reqs, table_stride, total_q, max_q_len,
                                                        1 if block_mass else 0)

    def attend(self, layer, q, block_table, kv_len, q_start=None, max_q_len=1, window=0, block_mass=None, out=None,
               scratch=None, stream=None):
        """Attend q [rows, Hq, D] (input dtype) over the pages; returns out of q's shape and
        type.  Without q_start there is one row per request; with it (int32 [n + 1], a
        plan's row_start) request r's rows are q_start[r] .. q_start[r + 1] - 1, its last
        tokens, at most max_q_len of them; rows behind the last request's are not written
        (a padded batch's are whatever was in memory).  window > 0: only the last `window` positions.
        block_mass: optional float32 [n, stride] that receives each visible block's mass
        (single-token rows only).  scratch: optional uint8 tensor of attend_scratch_bytes."""
        if stream is None and out is None and scratch is None and self._fast is not None:
            if _raw_stream(self._index) not in self._streams:
                self._mark(_raw_stream(self._index))
            r = self._fast.attend(self._key, layer, q, block_table, kv_len, q_start, max_q_len, window, block_mass)
            if r.__class__ is _Tensor:
                return r
            if r is not None:
                self._check(r)
        n, = self._need_dims(kv_len, "kv_len", _i32, 1)
        stride = self._need_dims(block_table, "block_table", _i32, 2)[1]
        rows = self._need_dims(q, "q", self.in_dtype, 3)[0]
        shape = (rows,) + self._qrow
        table = self._need(block_table, "block_table", _i32, (n, stride))
        qp = self._need(q, "q", self.in_dtype, shape)
        start = None if q_start is None else self._need(q_start, "q_start", _i32, (n + 1,))
        mass = None if block_mass is None else self._need(block_mass, "block_mass", _f32, (n, stride))
        if out is None:
            out = self._empty(shape, self.in_dtype, stream)
        op = self._need(out, "out", self.in_dtype, shape)
        if scratch is None:
            size = self.attend_scratch_bytes(n, stride, rows, max_q_len, mass is not None)
            scratch = self._empty((size,), torch.uint8, stream)
        else:
            size = scratch.numel()
            if (not scratch.is_cuda or scratch.device != self.device or scratch.dtype != torch.uint8
                    or not scratch.is_contiguous()):
                raise TypeError("scratch must be a contiguous uint8 tensor on %s" % self.device)
        st = self._lib.kvs_paged_attend(
            self._ctx, layer, n, table, stride, kv_len.data_ptr(), start, rows, max_q_len, window, qp, op, mass,
            scratch.data_ptr(), size, self._stream(stream))
        if st:
            self._check(st)
        return out

    # ---- inspection
    def get_status(self, stream=None):
        """Synchronise and return the device status code (0 = OK)."""
        return self._lib.kvs_paged_get_status(self._ctx, self._stream(stream))

    def clear_error(self, stream=None):
        self._check(self._lib.kvs_paged_clear_error(self._ctx, self._stream(stream)))

    def last_error(self):
        return self._lib.kvs_paged_last_error(self._ctx).decode()
