"""Thin ctypes binding of ``libpkv.so`` (the C ABI in ``include/pkv.h``).

Argument marshalling only: tensors become device pointers, lists of streams
become ``pkv_seq`` arrays, and the current torch CUDA stream is passed as the
launch stream.  Every step of the computation runs in the library's CUDA
kernels; there is no other path.  If the library is missing this module
raises instead of falling back to anything.
"""
from __future__ import annotations

import array
import ctypes
import os
import struct
from typing import Optional, Sequence

from . import build as _build

K, V, IK, P, KS, VS = 0, 1, 2, 3, 4, 5
KV_BF16, KV_E4M3 = 0, 1
OK, EINVAL, EAGAIN, ECUDA, EDEVICE = 0, 1, 2, 3, 4
DEV_BAD_PAGE, DEV_TIMEOUT, DEV_SMEM, DEV_RANGE = 1, 2, 4, 8
MAX_SEQS = 64
_NAMES = {EINVAL: "PKV_EINVAL", EAGAIN: "PKV_EAGAIN", ECUDA: "PKV_ECUDA", EDEVICE: "PKV_EDEVICE"}


class PkvError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {_NAMES.get(code, code)}")
        self.code = code


class Layout(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("idx_dim", ctypes.c_int32),
                ("kv_format", ctypes.c_int32)]


class Pg(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("page_elems", ctypes.c_int64), ("page_pos", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("n_table", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Seq(ctypes.Structure):
    _fields_ = [("pg", Pg), ("len", ctypes.c_int32), ("n_new", ctypes.c_int32)]


class EventOps(ctypes.Structure):
    RECORD = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                              ctypes.POINTER(ctypes.c_void_p))
    QUERY = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p)
    DESTROY = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_void_p)
    _fields_ = [("record", RECORD), ("query", QUERY), ("destroy", DESTROY),
                ("ctx", ctypes.c_void_p)]


_lib = None

EXPORTS = [
    "pkv_layout_page_elems", "pkv_pg_row", "pkv_arena_create", "pkv_arena_destroy",
    "pkv_arena_info", "pkv_pages_take", "pkv_pages_give", "pkv_arena_pg",
    "pkv_arena_set_event_ops", "pkv_run_pages", "pkv_run_take", "pkv_run_give", "pkv_run_map",
    "pkv_pages_fork", "pkv_pages_holders", "pkv_arena_compact", "pkv_pages_copy",
    "pkv_tables_remap", "pkv_store", "pkv_gather", "pkv_pool", "pkv_decode_ws_size",
    "pkv_decode", "pkv_decode_static", "pkv_block_scores", "pkv_topk", "pkv_sparse_ws_size",
    "pkv_sparse_decode", "pkv_prefill_ws_size", "pkv_prefill", "pkv_diag_wait_runs_out",
    "pkv_diag_cta_wait_runs_out", "pkv_window_decode_ws_size", "pkv_window_decode",
    "pkv_window_prefill_ws_size", "pkv_window_prefill", "pkv_window_dead_pages",
]


def library_path() -> str:
    return _build.LIB


def load(path: Optional[str] = None):
    """Load the CUDA library (built in-tree by ``build.build()``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with paged_kv_cache_pg_gb300.build.build()")
    lib = ctypes.CDLL(p)
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    LP, PP, SP = ctypes.POINTER(Layout), ctypes.POINTER(Pg), ctypes.POINTER(Seq)
    sig = {
        "pkv_layout_page_elems": [LP, i32, ctypes.POINTER(i64)],
        "pkv_pg_row": [LP, PP, vp, i32, i32, i32, i32, ctypes.POINTER(i64)],
        "pkv_arena_create": [LP, i32, vp, sz, ctypes.POINTER(vp)],
        "pkv_arena_destroy": [vp],
        "pkv_arena_info": [vp, ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.POINTER(i64)],
        "pkv_pages_take": [vp, i32, vp],
        "pkv_pages_give": [vp, vp, i32, vp, i32],
        "pkv_arena_pg": [vp, vp, i32, PP],
        "pkv_arena_set_event_ops": [vp, ctypes.POINTER(EventOps)],
        "pkv_pages_fork": [vp, vp, i32, i32, vp, ctypes.POINTER(i32), ctypes.POINTER(i32),
                           ctypes.POINTER(i32)],
        "pkv_pages_holders": [vp, vp, i32, vp],
        "pkv_arena_compact": [vp, i32, vp, vp, ctypes.POINTER(i32)],
        "pkv_pages_copy": [LP, i32, vp, i32, vp, vp, vp, i32, vp],
        "pkv_tables_remap": [vp, vp, i32, vp, vp, i32, vp],
        "pkv_run_pages": [vp, ctypes.c_uint64, ctypes.POINTER(i32)],
        "pkv_run_take": [vp, i32, ctypes.POINTER(i32)],
        "pkv_run_give": [vp, i32, i32, vp, i32],
        "pkv_run_map": [vp, i32, i32, vp, i32, ctypes.c_uint64, vp],
        "pkv_store": [LP, SP, i32, i32, vp, vp, vp, vp, vp],
        "pkv_gather": [LP, SP, i32, i32, i32, vp, vp, vp],
        "pkv_pool": [LP, SP, i32, i32, vp, vp],
        "pkv_decode_ws_size": [LP, SP, i32, i32, ctypes.POINTER(sz)],
        "pkv_decode": [LP, SP, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp, vp],
        "pkv_decode_static": [LP, SP, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp],
        "pkv_window_decode_ws_size": [LP, SP, i32, i32, i32, i32, ctypes.POINTER(sz)],
        "pkv_window_decode": [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp, vp],
        "pkv_window_prefill_ws_size": [LP, SP, i32, i32, i32, i32, ctypes.POINTER(sz)],
        "pkv_window_prefill": [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, sz, vp, vp],
        "pkv_window_dead_pages": [i32, i32, i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)],
        "pkv_prefill_ws_size": [LP, SP, i32, i32, ctypes.POINTER(sz)],
        "pkv_prefill": [LP, SP, i32, i32, i32, vp, vp, vp, sz, vp, vp],
        "pkv_block_scores": [LP, SP, i32, i32, i32, vp, vp, i32, vp, vp],
        "pkv_topk": [SP, i32, i32, vp, i32, i32, vp, vp],
        "pkv_sparse_ws_size": [LP, SP, i32, i32, i32, ctypes.POINTER(sz)],
        "pkv_sparse_decode": [LP, SP, i32, i32, i32, vp, vp, i32, vp, vp, sz, vp, vp],
        "pkv_diag_wait_runs_out": [vp, vp],
        "pkv_diag_cta_wait_runs_out": [vp, i32, vp],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise PkvError(rc, what)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_current = None  # (torch, the current device, its raw stream by device index), once torch is needed


def _torch_streams():
    global _current
    if _current is None:
        import torch
        # the raw handle without building a Stream object (about 3 us of a call)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        if torch.cuda.is_available():
            torch.cuda.init()
        else:
            device = lambda: -2   # of no tensor
        _current = (torch, device, raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))
    return _current


def _stream(stream) -> Optional[int]:
    if stream is None:
        _, device, raw = _current or _torch_streams()
        return raw(device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _seqs(seqs: Sequence[Seq]):
    if isinstance(seqs, ctypes.Array):
        return seqs, len(seqs)
    arr = (Seq * max(1, len(seqs)))(*seqs)
    return arr, len(seqs)


def _here(what: str, *tensors, dtype=None):
    """Device addresses of tensors that a kernel of the current device may
    touch as one block each: contiguous tensors on that device (of `dtype`
    when given); None and addresses given as ints are taken as they are."""
    dev, out = None, []
    for t in tensors:
        if t is not None and type(t) is not int:
            at = t.get_device()
            if dev is None and at >= 0:
                dev = (_current or _torch_streams())[1]()
            if at != dev or not t.is_contiguous() or (dtype is not None and t.dtype != dtype):
                raise PkvError(EINVAL, f"{what}: not a contiguous tensor of the type on the current device")
            t = t.data_ptr()
        out.append(t)
    return out


_counts = {}  # streams of a launch: reader of their new tokens
_types = None  # types of 16-bit rows; the status word's


def _window(what: str, lay, seqs, layer: int, n_q_heads: int, window: int, n_sink: int, q, out, ws, status, stream,
            chunk: bool, k=None, v=None, ik=None):
    """A windowed call.  Tensors have to be contiguous, on the current device, of
    the rows' type and as long as the launch's packed rows; rows given as ints
    (addresses) are taken as they are.  Written out for each tensor: a small
    call takes the GPU no longer than its arguments take here."""
    global _types
    if _types is None:
        torch = (_current or _torch_streams())[0]
        _types = frozenset((torch.bfloat16, torch.int16, torch.uint16)), torch.int32
    _ints(what, layer | n_q_heads | window | n_sink)
    arr, n = _seqs(seqs)
    if arr._type_ is not Seq:
        raise PkvError(EINVAL, f"{what}: the streams are not pkv_seq structures")
    read = _counts.get(n)
    if read is None:
        at = Seq.n_new.offset
        read = _counts[n] = struct.Struct("=" + f"{at}xi{ctypes.sizeof(Seq) - at - 4}x" * n).unpack_from
    new = read(arr)[0] if n == 1 else sum(read(arr)) if n else 0
    types, word = _types
    dev, ws_bytes, rows = (_current or _torch_streams())[1](), 0, 512 * n_q_heads * new
    if type(q) is not int and q is not None:
        if q.get_device() != dev or q.dtype not in types or q.nbytes < rows or not q.is_contiguous():
            _refuse(what, "q")
        q = q.data_ptr()
    if type(out) is not int and out is not None:
        if out.get_device() != dev or out.dtype not in types or out.nbytes < rows or not out.is_contiguous():
            _refuse(what, "out")
        out = out.data_ptr()
    if k is not None or v is not None:
        rows = 512 * lay.n_kv_heads * new
    if k is not None and type(k) is not int:
        if k.get_device() != dev or k.dtype not in types or k.nbytes < rows or not k.is_contiguous():
            _refuse(what, "k_new")
        k = k.data_ptr()
    if v is not None and type(v) is not int:
        if v.get_device() != dev or v.dtype not in types or v.nbytes < rows or not v.is_contiguous():
            _refuse(what, "v_new")
        v = v.data_ptr()
    if ik is not None and type(ik) is not int:
        if ik.get_device() != dev or ik.dtype not in types or ik.nbytes < 2 * lay.idx_dim * new or not ik.is_contiguous():
            _refuse(what, "ik_new")
        ik = ik.data_ptr()
    if ws is not None:  # (an address would say nothing of its size)
        if type(ws) is int or ws.get_device() != dev or not ws.is_contiguous():
            _refuse(what, "the workspace")
        ws_bytes, ws = ws.nbytes, ws.data_ptr()
    if status is not None and type(status) is not int:
        if status.get_device() != dev or status.dtype is not word or status.nbytes < 4:
            _refuse(what, "the status")
        status = status.data_ptr()
    lib, lay_at, seqs_at = load(), ctypes.addressof(lay), ctypes.addressof(arr)
    if chunk:
        rc = lib.pkv_window_prefill(lay_at, seqs_at, n, layer, n_q_heads, window, n_sink, q, out, ws, ws_bytes, status,
                                    _stream(stream))
    else:
        rc = lib.pkv_window_decode(lay_at, seqs_at, n, layer, n_q_heads, window, n_sink, q, k, v, ik, out, ws, ws_bytes,
                                   status, _stream(stream))
    _check(rc, what)


def _ints(what: str, bits: int):
    """Refuses what is negative or not a 32-bit integer (`bits`: all of them, or-ed),
    which ctypes would cut to its low 32 bits."""
    if bits >> 31:
        raise PkvError(EINVAL, f"{what}: an integer that is negative or beyond 32 bits")


def _refuse(what: str, name: str):
    raise PkvError(EINVAL, f"{what}: {name} is not a contiguous tensor of its type, long enough, on the current device")


_np = _i32 = None


def _host_i32(what: str, a):
    """Host integers as int32: how many, and their bytes (which ctypes passes
    as an address, sooner than it finds an array's).  Refuses a value that is
    not a 32-bit integer."""
    global _np, _i32
    if _np is None:
        import numpy
        _np, _i32 = numpy, numpy.dtype(numpy.int32)
    if type(a) is not _np.ndarray or a.dtype is not _i32:
        given = _np.asarray(a)
        with _np.errstate(invalid="ignore"):
            a = given.astype(_np.int32)
        if not _np.array_equal(a, given):
            raise PkvError(EINVAL, f"{what}: not 32-bit integers")
    return a.size, a.tobytes()


# ---- descriptors ------------------------------------------------------------

def layout(n_layers: int, n_kv_heads: int, head_dim: int = 256, idx_dim: int = 128,
           kv_format: int = KV_BF16) -> Layout:
    """kv_format KV_E4M3: K and V rows are e4m3 codes + a float32 scale each."""
    return Layout(n_layers, n_kv_heads, head_dim, idx_dim, kv_format)


def page_elems(lay: Layout, page_pos: int) -> int:
    out = ctypes.c_int64()
    _check(load().pkv_layout_page_elems(ctypes.byref(lay), page_pos, ctypes.byref(out)),
           "pkv_layout_page_elems")
    return out.value


def pg(base, table, page_elems_: int, page_pos: int, n_pages: int = 1,
       n_table: Optional[int] = None) -> Pg:
    """A stream's Pg: table None means a contiguous buffer of page_pos rows a head."""
    if table is None:
        return Pg(_ptr(base), None, page_elems_, page_pos, 1, 1, 0)
    nt = int(table.numel()) if n_table is None else n_table
    return Pg(_ptr(base), _ptr(table), page_elems_, page_pos, n_pages, nt, 0)


def seq(pg_: Pg, length: int, n_new: int) -> Seq:
    return Seq(pg_, length, n_new)


def batch(seqs: Sequence[Seq]):
    """The streams of a launch as one ctypes array, for programs that keep it
    between calls (its entries' len and n_new may be changed in place).  Every
    call that takes a list of streams takes it as well."""
    return (Seq * len(seqs))(*seqs)


def pg_row(lay: Layout, pg_: Pg, host_table, layer: int, kind: int, head: int, pos: int) -> int:
    """Host pg_at: element offset of a row from pg.base; host_table is a numpy int32 array."""
    out = ctypes.c_int64()
    tab = None if host_table is None else host_table.ctypes.data
    _check(load().pkv_pg_row(ctypes.byref(lay), ctypes.byref(pg_), tab, layer, kind, head, pos,
                             ctypes.byref(out)), "pkv_pg_row")
    return out.value


class Arena:
    """The page pool over caller-owned device memory (a torch tensor)."""

    def __init__(self, lay: Layout, page_pos: int, memory, nbytes: Optional[int] = None):
        self._lib = load()
        self._h = ctypes.c_void_p()
        self.memory = memory
        n = nbytes if nbytes is not None else memory.numel() * memory.element_size()
        _check(self._lib.pkv_arena_create(ctypes.byref(lay), page_pos, _ptr(memory), n,
                                          ctypes.byref(self._h)), "pkv_arena_create")
        self._ops = None

    def close(self):
        if self._h:
            self._lib.pkv_arena_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def info(self):
        n, f, e = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
        _check(self._lib.pkv_arena_info(self._h, ctypes.byref(n), ctypes.byref(f),
                                        ctypes.byref(e)), "pkv_arena_info")
        return n.value, f.value, e.value

    def take(self, n: int):
        import numpy as np
        ids = np.zeros(max(1, n), dtype=np.int32)
        _check(self._lib.pkv_pages_take(self._h, n, ids.ctypes.data), "pkv_pages_take")
        return ids[:n]

    def give(self, ids, stream=None, defer: bool = True):
        import numpy as np
        ids = np.ascontiguousarray(ids, dtype=np.int32)
        st = _stream(stream) if defer else (stream or 0)
        _check(self._lib.pkv_pages_give(self._h, ids.ctypes.data, ids.size, st, int(defer)),
               "pkv_pages_give")

    def fork(self, ids, length: int):
        """Share a stream's pages with a new one: (its ids, copy), where copy
        is None or (src, dst, n_pos) of the last page, which is its own."""
        import numpy as np
        _ints("pkv_pages_fork", length)
        n_ids, ids = _host_i32("pkv_pages_fork", ids)
        out = np.empty(max(1, n_ids), dtype=np.int32)
        s, d, n = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check(self._lib.pkv_pages_fork(self._h, ids, n_ids, length, out.ctypes.data,
                                        ctypes.byref(s), ctypes.byref(d), ctypes.byref(n)),
               "pkv_pages_fork")
        return out[:n_ids], ((s.value, d.value, n.value) if n.value else None)

    def holders(self, ids):
        import numpy as np
        n, ids = _host_i32("pkv_pages_holders", ids)
        out = np.zeros(max(1, n), dtype=np.int32)
        _check(self._lib.pkv_pages_holders(self._h, ids, n, out.ctypes.data), "pkv_pages_holders")
        return out[:n]

    def compact(self, max_moves: int):
        """Plan up to max_moves moves of high pages to low holes: (src, dst).
        The caller copies the pages, rewrites the tables and gives src back."""
        import numpy as np
        _ints("pkv_arena_compact", max_moves)
        src, dst = (np.zeros(max(1, max_moves), dtype=np.int32) for _ in range(2))
        n = ctypes.c_int32()
        _check(self._lib.pkv_arena_compact(self._h, max_moves, src.ctypes.data, dst.ctypes.data,
                                           ctypes.byref(n)), "pkv_arena_compact")
        return src[:n.value], dst[:n.value]

    def run_pages(self, run_bytes: int) -> int:
        k = ctypes.c_int32()
        _check(self._lib.pkv_run_pages(self._h, run_bytes, ctypes.byref(k)), "pkv_run_pages")
        return k.value

    def run_take(self, k: int) -> int:
        first = ctypes.c_int32()
        _check(self._lib.pkv_run_take(self._h, k, ctypes.byref(first)), "pkv_run_take")
        return first.value

    def run_give(self, first: int, k: int, stream=None, defer: bool = True):
        st = _stream(stream) if defer else (stream or 0)
        _check(self._lib.pkv_run_give(self._h, first, k, st, int(defer)), "pkv_run_give")

    def run_map(self, first: int, k: int, part_bytes, align: int = 256):
        """Device addresses of the parts laid one after another in the run."""
        import numpy as np
        parts = np.ascontiguousarray(part_bytes, dtype=np.uint64)
        out = (ctypes.c_void_p * max(1, parts.size))()
        _check(self._lib.pkv_run_map(self._h, first, k, parts.ctypes.data, parts.size, align,
                                     out), "pkv_run_map")
        return [int(out[i] or 0) for i in range(parts.size)]

    def pg(self, dev_table, n_table: Optional[int] = None) -> Pg:
        out = Pg()
        nt = int(dev_table.numel()) if n_table is None else n_table
        _check(self._lib.pkv_arena_pg(self._h, _ptr(dev_table), nt, ctypes.byref(out)),
               "pkv_arena_pg")
        return out

    def set_event_ops(self, ops: Optional[EventOps]):
        self._ops = ops
        _check(self._lib.pkv_arena_set_event_ops(self._h, ctypes.byref(ops) if ops else None),
               "pkv_arena_set_event_ops")


# ---- kernels ------------------------------------------------------------------

def store(lay, seqs, layer, k_new, v_new, ik_new=None, status=None, stream=None):
    arr, n = _seqs(seqs)
    _check(load().pkv_store(ctypes.byref(lay), arr, n, layer, _ptr(k_new), _ptr(v_new),
                            _ptr(ik_new), _ptr(status), _stream(stream)), "pkv_store")


def gather(lay, seqs, layer, kind, out, status=None, stream=None):
    arr, n = _seqs(seqs)
    _check(load().pkv_gather(ctypes.byref(lay), arr, n, layer, kind, _ptr(out), _ptr(status),
                             _stream(stream)), "pkv_gather")


def pages_copy(lay, page_pos: int, memory, n_pages: int, src, dst, n_pos=None, stream=None):
    """Copy pages src[i] to dst[i] of the arena at `memory`, whole or their
    first n_pos[i] positions; src, dst, n_pos: host integers."""
    (n, src), (n_dst, dst) = _host_i32("pkv_pages_copy", src), _host_i32("pkv_pages_copy", dst)
    n_n_pos, n_pos = (n, None) if n_pos is None else _host_i32("pkv_pages_copy", n_pos)
    if n_dst != n or n_n_pos != n:
        raise PkvError(EINVAL, "pkv_pages_copy: lists of different lengths")
    _ints("pkv_pages_copy", page_pos | n_pages)
    base, = _here("pkv_pages_copy", memory)
    if base is not memory and memory.nbytes < 2 * n_pages * page_elems(lay, page_pos):
        raise PkvError(EINVAL, "pkv_pages_copy: the memory holds fewer pages")
    _check(load().pkv_pages_copy(ctypes.byref(lay), page_pos, base, n_pages, src, dst, n_pos, n,
                                 _stream(stream)), "pkv_pages_copy")


def tables_remap(tables, src, dst, stream=None):
    """Rewrite device page tables after a compaction: entries src[i] become
    dst[i].  tables: int32 device tensors; src, dst: host integers."""
    (n_moves, src), (n_dst, dst) = _host_i32("pkv_tables_remap", src), _host_i32("pkv_tables_remap", dst)
    if n_moves != n_dst:
        raise PkvError(EINVAL, "pkv_tables_remap: lists of different lengths")
    torch = (_current or _torch_streams())[0]
    n = len(tables)
    if any(type(t) is int for t in tables):
        raise PkvError(EINVAL, "pkv_tables_remap: the tables are tensors")
    ptrs = array.array("Q", _here("pkv_tables_remap", *tables, dtype=torch.int32)).tobytes()
    sizes = array.array("i", [t.numel() for t in tables]).tobytes()
    _check(load().pkv_tables_remap(ptrs, sizes, n, src, dst, n_moves, _stream(stream)),
           "pkv_tables_remap")


def pool(lay, seqs, layer, status=None, stream=None):
    arr, n = _seqs(seqs)
    _check(load().pkv_pool(ctypes.byref(lay), arr, n, layer, _ptr(status), _stream(stream)),
           "pkv_pool")


def decode_ws_size(lay, seqs, n_q_heads) -> int:
    arr, n = _seqs(seqs)
    out = ctypes.c_size_t()
    _check(load().pkv_decode_ws_size(ctypes.byref(lay), arr, n, n_q_heads, ctypes.byref(out)),
           "pkv_decode_ws_size")
    return out.value


def decode(lay, seqs, layer, n_q_heads, q, out, ws, status=None, stream=None, k_new=None,
           v_new=None, ik_new=None):
    """Decode attention; with k_new/v_new (and ik_new) the new rows are stored too."""
    arr, n = _seqs(seqs)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().pkv_decode(ctypes.byref(lay), arr, n, layer, n_q_heads, _ptr(q), _ptr(k_new),
                             _ptr(v_new), _ptr(ik_new), _ptr(out), _ptr(ws), ws_bytes,
                             _ptr(status), _stream(stream)), "pkv_decode")


def prefill_ws_size(lay, seqs, n_q_heads) -> int:
    arr, n = _seqs(seqs)
    out = ctypes.c_size_t()
    _check(load().pkv_prefill_ws_size(ctypes.byref(lay), arr, n, n_q_heads, ctypes.byref(out)),
           "pkv_prefill_ws_size")
    return out.value


def prefill(lay, seqs, layer, n_q_heads, q, out, ws, status=None, stream=None):
    """Chunked-prefill attention on the tensor cores (the chunk already stored)."""
    arr, n = _seqs(seqs)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().pkv_prefill(ctypes.byref(lay), arr, n, layer, n_q_heads, _ptr(q), _ptr(out),
                              _ptr(ws), ws_bytes, _ptr(status), _stream(stream)), "pkv_prefill")


def window_decode_ws_size(lay, seqs, n_q_heads, window, n_sink) -> int:
    _ints("pkv_window_decode_ws_size", n_q_heads | window | n_sink)
    arr, n = _seqs(seqs)
    out = ctypes.c_size_t()
    _check(load().pkv_window_decode_ws_size(ctypes.byref(lay), arr, n, n_q_heads, window, n_sink,
                                            ctypes.byref(out)), "pkv_window_decode_ws_size")
    return out.value


def window_decode(lay, seqs, layer, n_q_heads, window, n_sink, q, out, ws=None, status=None,
                  stream=None, k_new=None, v_new=None, ik_new=None):
    """Decode attention over the newest `window` positions and the first
    n_sink; with k_new/v_new (and ik_new) the new rows are stored too."""
    _window("pkv_window_decode", lay, seqs, layer, n_q_heads, window, n_sink, q, out, ws, status, stream, False,
            k_new, v_new, ik_new)


def window_prefill_ws_size(lay, seqs, n_q_heads, window, n_sink) -> int:
    _ints("pkv_window_prefill_ws_size", n_q_heads | window | n_sink)
    arr, n = _seqs(seqs)
    out = ctypes.c_size_t()
    _check(load().pkv_window_prefill_ws_size(ctypes.byref(lay), arr, n, n_q_heads, window, n_sink,
                                             ctypes.byref(out)), "pkv_window_prefill_ws_size")
    return out.value


def window_prefill(lay, seqs, layer, n_q_heads, window, n_sink, q, out, ws, status=None,
                   stream=None):
    """Chunk attention on the tensor cores over the newest `window` positions
    of each query and the first n_sink (the chunk already stored)."""
    _window("pkv_window_prefill", lay, seqs, layer, n_q_heads, window, n_sink, q, out, ws, status, stream, True)


def window_dead_pages(page_pos: int, length: int, window: int, n_sink: int):
    """Logical pages [first, end) that no query at position `length` or later reads."""
    _ints("pkv_window_dead_pages", page_pos | length | window | n_sink)
    first, end = ctypes.c_int32(), ctypes.c_int32()
    _check(load().pkv_window_dead_pages(page_pos, length, window, n_sink, ctypes.byref(first),
                                        ctypes.byref(end)), "pkv_window_dead_pages")
    return first.value, end.value


STATIC_SCRATCH_BYTES = 4 << 20


def decode_static(lay, seqs, layer, n_q_heads, q, out, status=None, stream=None, k_new=None,
                  v_new=None, ik_new=None):
    """pkv_decode without a workspace: for callers that cannot allocate device
    memory.  The partials go to a fixed 4 MiB array inside the library; calls
    that run at the same time on the GPU share it, so issue them in order."""
    arr, n = _seqs(seqs)
    _check(load().pkv_decode_static(ctypes.byref(lay), arr, n, layer, n_q_heads, _ptr(q),
                                    _ptr(k_new), _ptr(v_new), _ptr(ik_new), _ptr(out),
                                    _ptr(status), _stream(stream)), "pkv_decode_static")


def block_scores(lay, seqs, layer, n_q_heads, qi, scores, ld, status=None, stream=None):
    arr, n = _seqs(seqs)
    _check(load().pkv_block_scores(ctypes.byref(lay), arr, n, layer, n_q_heads, _ptr(qi),
                                   _ptr(scores), ld, _ptr(status), _stream(stream)),
           "pkv_block_scores")


def topk(seqs, n_q_heads, scores, ld, k, ids, stream=None):
    arr, n = _seqs(seqs)
    _check(load().pkv_topk(arr, n, n_q_heads, _ptr(scores), ld, k, _ptr(ids), _stream(stream)),
           "pkv_topk")


def sparse_ws_size(lay, seqs, n_q_heads, k) -> int:
    arr, n = _seqs(seqs)
    out = ctypes.c_size_t()
    _check(load().pkv_sparse_ws_size(ctypes.byref(lay), arr, n, n_q_heads, k,
                                     ctypes.byref(out)), "pkv_sparse_ws_size")
    return out.value


def sparse_decode(lay, seqs, layer, n_q_heads, q, ids, k, out, ws, status=None, stream=None):
    arr, n = _seqs(seqs)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().pkv_sparse_decode(ctypes.byref(lay), arr, n, layer, n_q_heads, _ptr(q),
                                    _ptr(ids), k, _ptr(out), _ptr(ws), ws_bytes, _ptr(status),
                                    _stream(stream)), "pkv_sparse_decode")


def diag_wait_runs_out(status, stream=None):
    """One warp's wait on a barrier nothing arrives on: it gives up after about
    a second and sets PKV_DEV_TIMEOUT in `status` (a device int32)."""
    _check(load().pkv_diag_wait_runs_out(_ptr(status), _stream(stream)), "pkv_diag_wait_runs_out")


def diag_cta_wait_runs_out(status, withheld_slice=2, stream=None):
    """A decode-shaped CTA (eight warps, four key slices, twelve stage slots)
    in which one slice's stage never lands: that slice's waits give up after
    about a second, the CTA returns as a whole and PKV_DEV_TIMEOUT is set in
    `status` (a device int32)."""
    _check(load().pkv_diag_cta_wait_runs_out(_ptr(status), withheld_slice, _stream(stream)),
           "pkv_diag_cta_wait_runs_out")
