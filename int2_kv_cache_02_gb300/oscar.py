"""Python binding of liboscar (include/oscar.h): argument marshalling only.

Every computation runs in the CUDA kernels of liboscar.so; this module turns
torch tensors into device pointers, keeps the oscar_cache struct, and raises
OscarError on a non-OK status.  Importing it fails loudly if the library has
not been built (``__graft_entry__.build()`` or ``python -m
int2_kv_cache_02_gb300._build``): there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from ctypes import POINTER, c_float, c_int, c_longlong, c_size_t, c_uint, c_ulonglong, c_void_p

import torch

from . import _build

D, G, R = 128, 32, 128
NO_ROTATE, NO_SCALE, NORM_ALL_HEADS = 1, 2, 4

_STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "ALIGNMENT", 4: "CAPACITY",
           5: "WORKSPACE", 6: "CUDA", 7: "DEVICE_STATUS"}


class OscarError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)} "
                         f"({_lib.oscar_status_string(status).decode()})")


class OscarCacheStruct(ctypes.Structure):
    _fields_ = [("B", c_int), ("Hkv", c_int), ("T_cap", c_int),
                ("packed", c_void_p),
                ("k_res", c_void_p), ("v_res", c_void_p), ("k_res_norm", c_void_p),
                ("n_packed", c_int), ("n_res", c_int), ("flags", c_uint),
                ("norm_target", c_float), ("key_group", c_int), ("bits", c_int)]


class OscarPagedCacheStruct(ctypes.Structure):
    _fields_ = [("B", c_int), ("Hkv", c_int), ("max_blocks", c_int), ("n_pages", c_int),
                ("pages", c_void_p), ("block_table", c_void_p),
                ("n_packed", c_void_p), ("n_res", c_void_p),
                ("k_res", c_void_p), ("v_res", c_void_p), ("k_res_norm", c_void_p),
                ("flags", c_uint), ("norm_target", c_float), ("key_group", c_int),
                ("bits", c_int)]


class OscarKV16CacheStruct(ctypes.Structure):
    _fields_ = [("B", c_int), ("Hkv", c_int), ("max_blocks", c_int), ("n_pages", c_int),
                ("T_cap", c_int), ("dtype", c_int),
                ("k", c_void_p), ("v", c_void_p), ("weight", c_void_p),
                ("block_table", c_void_p), ("n_tok", c_void_p)]


BLOCK_BYTES = 2752
BLOCK_BYTES_INT4 = 4800
# byte ranges of the fields of one 32-token block record (include/oscar.h)
RECORD_FIELDS = {"k_codes": (0, 1024), "v_codes": (1024, 2048), "k_scale": (2048, 2304),
                 "k_zero": (2304, 2560), "k_norm": (2560, 2624), "v_scale": (2624, 2688),
                 "v_zero": (2688, 2752)}
# the INT4 record: twice the code bytes, the same side arrays after them
RECORD_FIELDS_INT4 = {"k_codes": (0, 2048), "v_codes": (2048, 4096), "k_scale": (4096, 4352),
                      "k_zero": (4352, 4608), "k_norm": (4608, 4672), "v_scale": (4672, 4736),
                      "v_zero": (4736, 4800)}
PER_TOKEN_FIELDS = ("k_norm", "v_scale", "v_zero")
_KV16_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


def record_bytes(bits: int = 2) -> int:
    return BLOCK_BYTES_INT4 if bits == 4 else BLOCK_BYTES


def _load() -> ctypes.CDLL:
    path = _build.lib_path("liboscar.so")
    if not os.path.exists(path):
        raise ImportError(f"liboscar.so is not built ({path}); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P = POINTER(OscarCacheStruct)
    PP = POINTER(OscarPagedCacheStruct)
    P16 = POINTER(OscarKV16CacheStruct)
    sig = {
        "oscar_rotate_q": (c_int, [c_void_p, c_void_p, c_int, c_int, c_uint, c_void_p]),
        "oscar_rotate_scale_k": (c_int, [c_void_p, c_int, c_void_p, c_void_p, c_int, c_int,
                                         c_int, c_int, c_int, c_uint, c_float, c_void_p]),
        "oscar_quantize_kv": (c_int, [P, c_void_p, c_void_p, c_void_p, c_int, c_int, c_void_p]),
        "oscar_append_kv": (c_int, [P, c_void_p, c_void_p, c_int, c_void_p]),
        "oscar_prefill_kv": (c_int, [P, c_void_p, c_void_p, c_int, c_int, c_void_p]),
        "oscar_paged_prefill_kv": (c_int, [PP, c_void_p, c_void_p, c_int, c_void_p, c_int,
                                           c_void_p]),
        "oscar_paged_append_kv": (c_int, [PP, c_void_p, c_void_p, c_void_p, c_void_p]),
        "oscar_paged_decode_attention": (c_int, [PP, c_void_p, c_int, c_float, c_int, c_void_p,
                                                 c_int, c_void_p, c_size_t, c_void_p]),
        "oscar_decode_attention": (c_int, [P, c_void_p, c_int, c_float, c_void_p, c_int,
                                           c_void_p, c_size_t, c_void_p]),
        "oscar_decode_attention_static_ws": (c_int, [P, c_void_p, c_int, c_float, c_void_p,
                                                     c_int, c_void_p]),
        "oscar_decode_step": (c_int, [P, c_void_p, c_void_p, c_void_p, c_int, c_float, c_void_p,
                                      c_int, c_void_p, c_size_t, c_void_p]),
        "oscar_decode_num_splits": (c_int, [c_int, c_int, c_int, c_int]),
        "oscar_decode_plan_splits": (c_int, [ctypes.c_longlong, ctypes.c_longlong, c_int, c_int]),
        "oscar_decode_workspace_bytes": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
        "oscar_bf16_decode_attention": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int,
                                                c_int, c_int, c_int, c_float, c_void_p, c_int,
                                                c_void_p, c_size_t, c_void_p]),
        "oscar_kv16_write": (c_int, [P16, c_void_p, c_longlong, c_void_p, c_longlong, c_void_p,
                                     c_void_p, c_int, c_void_p]),
        "oscar_kv16_attention": (c_int, [P16, c_void_p, c_longlong, c_void_p, c_int, c_int,
                                         c_float, c_int, c_int, c_int, c_void_p, c_void_p,
                                         c_void_p, c_size_t, c_void_p]),
        "oscar_kv16_attention_workspace_bytes": (c_size_t, [P16, c_int, c_int, c_int, c_int,
                                                            c_int]),
        "oscar_kv16_decode_attention": (c_int, [P16, c_void_p, c_longlong, c_int, c_float, c_int,
                                                c_int, c_int, c_int, c_void_p, c_void_p,
                                                c_size_t, c_void_p]),
        "oscar_kv16_decode_workspace_bytes": (c_size_t, [P16, c_int, c_int, c_int, c_int,
                                                         c_int]),
        "oscar_kv16_accumulate": (c_int, [P16, c_void_p, c_longlong, c_void_p, c_void_p, c_int,
                                          c_int, c_float, c_int, c_int, c_int, c_int, c_void_p]),
        "oscar_kv16_evict": (c_int, [P16, P16, c_int, c_int, c_int, c_int, c_void_p, c_void_p,
                                     c_size_t, c_void_p]),
        "oscar_kv16_evict_workspace_bytes": (c_size_t, [P16, c_int, c_int, c_int, c_int]),
        "oscar_kv16_shared_decode_attention": (c_int, [P16, c_void_p, c_longlong, c_int, c_void_p,
                                                       c_void_p, c_int, c_float, c_int, c_int,
                                                       c_int, c_void_p, c_void_p, c_size_t,
                                                       c_void_p]),
        "oscar_kv16_shared_decode_workspace_bytes": (c_size_t, [P16, c_int, c_int, c_int, c_int,
                                                                c_int]),
        "oscar_kv16_shared_attention": (c_int, [P16, c_void_p, c_longlong, c_void_p, c_int, c_int,
                                                c_void_p, c_void_p, c_int, c_float, c_int, c_int,
                                                c_int, c_void_p, c_void_p, c_void_p, c_size_t,
                                                c_void_p]),
        "oscar_kv16_shared_attention_workspace_bytes": (c_size_t, [P16, c_int, c_int, c_int, c_int,
                                                                   c_int, c_int]),
        "oscar_kv16_fork": (c_int, [P16, P16, c_void_p, c_int, c_int, c_void_p]),
        "oscar_page_compact": (c_int, [c_void_p, c_void_p, c_int, c_int, c_int, c_void_p, c_void_p,
                                       c_void_p, c_size_t, c_void_p]),
        "oscar_page_compact_workspace_bytes": (c_size_t, [c_int, c_int, c_int]),
        "oscar_kv16_copy_pages": (c_int, [P16, P16, c_void_p, c_void_p, c_int, c_void_p]),
        "oscar_paged_copy_pages": (c_int, [PP, c_void_p, c_void_p, c_int, c_void_p]),
        "oscar_device_status": (c_int, [c_void_p]),
        "oscar_selftest_wait_timeout": (c_int, [c_uint, c_void_p]),
        "oscar_selftest_tc_wait_timeout": (c_int, [c_uint, c_void_p, c_void_p]),
        "oscar_selftest_kv16_decode_timeout": (c_int, [P16, c_void_p, c_int, c_int, c_void_p,
                                                       c_void_p, c_size_t, c_void_p]),
        "oscar_selftest_kv16_shared_timeout": (c_int, [P16, c_void_p, c_int, c_void_p, c_void_p,
                                                       c_int, c_int, c_int, c_void_p, c_void_p,
                                                       c_size_t, c_void_p]),
        "oscar_status_string": (ctypes.c_char_p, [c_int]),
        "oscar_kernel_launches": (c_ulonglong, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    return _lib


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("liboscar takes device tensors")
    if not t.is_contiguous():
        raise ValueError("liboscar takes contiguous tensors")
    return c_void_p(t.data_ptr())


def _stream(stream) -> c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _capturing(stream, device) -> bool:
    """Is `stream` (None: the device's current one) being captured into a graph?"""
    if device.type != "cuda":
        return False
    if stream is None and torch._C._cuda_getDevice() == device.index:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(device):
        if stream is None:
            return torch.cuda.is_current_stream_capturing()
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            return torch.cuda.is_current_stream_capturing()


def _check(st: int, where: str):
    if st != 0:
        raise OscarError(st, where)


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------

class KVCache:
    """Caller-owned device buffers of one layer's OScaR cache plus the
    oscar_cache struct that points at them (layouts in include/oscar.h)."""

    def __init__(self, B: int, Hkv: int, T_cap: int, flags: int = 0, device=None,
                 norm_target: float = 0.0, key_group: int = 0, bits: int = 0):
        if T_cap % G:
            raise ValueError("T_cap must be a multiple of 32")
        dev = torch.device(device if device is not None else "cuda")
        self.packed = torch.zeros((B, Hkv, T_cap // G, record_bytes(bits)), dtype=torch.uint8,
                                  device=dev)
        self.k_res = torch.zeros((B, Hkv, R, D), dtype=torch.bfloat16, device=dev)
        self.v_res = torch.zeros((B, Hkv, R, D), dtype=torch.bfloat16, device=dev)
        self.k_res_norm = torch.zeros((B, Hkv, R), dtype=torch.float16, device=dev)
        s = OscarCacheStruct()
        s.B, s.Hkv, s.T_cap = B, Hkv, T_cap
        for name in ("packed", "k_res", "v_res", "k_res_norm"):
            setattr(s, name, getattr(self, name).data_ptr())
        s.n_packed, s.n_res, s.flags, s.norm_target = 0, 0, flags, norm_target
        s.key_group = key_group
        s.bits = bits
        self.struct = s

    B = property(lambda self: self.struct.B)
    Hkv = property(lambda self: self.struct.Hkv)
    T_cap = property(lambda self: self.struct.T_cap)
    n_packed = property(lambda self: self.struct.n_packed)
    n_res = property(lambda self: self.struct.n_res)
    flags = property(lambda self: self.struct.flags)
    norm_target = property(lambda self: self.struct.norm_target)
    key_group = property(lambda self: self.struct.key_group or 32)
    bits = property(lambda self: self.struct.bits or 2)

    def ref(self):
        return ctypes.byref(self.struct)

    def field(self, name: str) -> torch.Tensor:
        """Writable view of one record field for every block:
        [B][Hkv][T_cap/32][n] with n = 256 words (codes; INT4: 512) or 128 halves (key
        step / zero); the per-token arrays (k_norm, v_scale, v_zero) as
        [B][Hkv][T_cap/32][4][8], element [j][i] = token 8j + i of the block."""
        lo, hi = (RECORD_FIELDS_INT4 if self.bits == 4 else RECORD_FIELDS)[name]
        raw = self.packed[..., lo:hi]
        if name.endswith("codes"):
            return raw.view(torch.int32)
        f = raw.view(torch.float16)
        if name in PER_TOKEN_FIELDS:
            # stored at 4 (t % 8) + t // 8: an [8][4] array, read transposed
            return f.unflatten(-1, (8, 4)).transpose(-1, -2)
        return f

    def tokens(self, name: str) -> torch.Tensor:
        """A copy of a field in token order: key codes [B][Hkv][T_cap][8]
        (INT4: [..][16]); norms and value step / zero [B][Hkv][T_cap]; value
        codes and key step / zero stay per block ([B][Hkv][T_cap/32][n])."""
        f = self.field(name)
        if name == "k_codes":
            return f.reshape(self.B, self.Hkv, self.T_cap, 4 * self.bits)
        if name in PER_TOKEN_FIELDS:
            return f.reshape(self.B, self.Hkv, self.T_cap)
        return f.clone()

    def nbytes(self) -> int:
        return sum(getattr(self, n).numel() * getattr(self, n).element_size()
                   for n in ("packed", "k_res", "v_res", "k_res_norm"))


class _PagePool:
    """Host-side page allocator of the paged caches: which pages are free, how
    many table entries name each of the others, and the block table's host copy
    beside the device's (self.block_table).  The table is written by these calls
    and by kv16_fork (share); entries in tables that a caller makes over the same
    pages are not counted.  Not while the current stream is captured into a graph."""

    def _init_pool(self, B: int, max_blocks: int, n_pages: int):
        self._behind = self._replayed = False
        self._free = list(range(n_pages))
        self._named = [0] * n_pages
        self._table_host = [[-1] * max_blocks for _ in range(B)]

    def _table_written(self, stream):
        """A call that writes the table has been queued on the stream, or captured:
        then any replay writes it again."""
        self._behind = True
        self._replayed |= _capturing(stream, self.block_table.device)

    def _follow(self, changes: bool = True):
        """Where a fork has written the table: waits for the device, and the host's
        copy, the counts and the free pages go by what the table says now.  `changes`:
        of the calls that change them, which a replayed graph would not repeat."""
        if (changes or self._behind) and _capturing(None, self.block_table.device):
            raise RuntimeError(f"{type(self).__name__}: the page allocator works on the host, "
                               "which a captured graph does not")
        if not self._behind:
            return
        table, n = self.block_table, len(self._named)
        if table.is_cuda:
            torch.cuda.synchronize(table.device)
        rows, named = [[p if p < n else -1 for p in row] for row in table.tolist()], [0] * n
        for row in rows:
            for p in row:
                if p >= 0:
                    named[p] += 1
        self._free = [p for p in self._free if not named[p]] + \
            [p for p in range(n) if self._named[p] and not named[p]]
        self._table_host, self._named, self._behind = rows, named, self._replayed

    def map_blocks(self, b: int, n_blocks: int, order=None):
        """Gives sequence b pages for its logical blocks 0..n_blocks-1 (those
        not mapped yet), taking free pages in `order` (a permutation of page
        ids, for tests) or those that have been free longest first.  A pool with
        too few of them gives none."""
        self._follow()
        row = self._table_host[b]
        missing = [j for j in range(n_blocks) if row[j] < 0]
        if len(missing) > len(self._free):
            raise OscarError(4, f"{type(self).__name__}.map_blocks: page pool exhausted")
        if order is not None:
            free = set(self._free)
            self._free = [p for p in order if p in free]
        for j in missing:
            row[j] = self._free.pop(0)
            self._named[row[j]] = 1
        self.block_table[b].copy_(torch.tensor(row, dtype=torch.int32))

    def share_blocks(self, b: int, parent: int, n_blocks: int):
        """Lets sequence b's logical blocks 0..n_blocks-1 be the pages of sequence
        parent's; those that b had there are given back.  Whole pages only: what
        is written to a shared page reaches every sequence that has it."""
        self._follow()
        row, theirs = self._table_host[b], self._table_host[parent]
        if not 0 <= n_blocks <= len(row) or any(p < 0 for p in theirs[:n_blocks]):
            raise OscarError(1, f"{type(self).__name__}.share_blocks: sequence {parent} has no "
                                f"{n_blocks} blocks")
        for j in range(n_blocks):
            if row[j] == theirs[j]:
                continue
            self._named[theirs[j]] += 1
            self._give_back(row, j)
            row[j] = theirs[j]
        self.block_table[b].copy_(torch.tensor(row, dtype=torch.int32))

    def _give_back(self, row: list, j: int):
        page, row[j] = row[j], -1
        if page >= 0:
            self._named[page] -= 1
            if self._named[page] == 0:
                self._free.append(page)

    def compact(self):
        """Gives the pages in use the lowest ids (page_compact): the table and the
        allocator go by the new ids from here on.  Returns (moves, counts) for
        the copies (kv16_copy_pages, paged_copy_pages), which come next on the
        current stream."""
        self._follow()
        table, n_pages = self.block_table, len(self._named)
        moves = torch.empty((n_pages // 2, 2), dtype=torch.int32, device=table.device)
        counts = torch.empty(2, dtype=torch.int32, device=table.device)
        workspace = alloc_workspace(page_compact_workspace_bytes(table, n_pages), table.device)
        page_compact(table, table, n_pages, moves, counts, workspace)
        # the same rule on the host's copy
        live = sum(n > 0 for n in self._named)
        old = [p for p in range(live, n_pages) if self._named[p]]
        to = dict(zip(old, [p for p in range(live) if not self._named[p]]))
        self._table_host = [[to.get(p, p) for p in row] for row in self._table_host]
        for p, q in to.items():
            self._named[q], self._named[p] = self._named[p], 0
        self._free = list(range(live, n_pages))
        return moves, counts

    def page_of(self, b: int, block: int) -> int:
        self._follow(changes=False)
        return self._table_host[b][block]

    def release_blocks(self, b: int, n_blocks: int = 0):
        """Takes back sequence b's pages behind its first n_blocks logical
        blocks; those that no other sequence shares are free for any sequence
        from then on, so work that reads them has to be queued before what
        writes them."""
        self._follow()
        row = self._table_host[b]
        for j in range(n_blocks, len(row)):
            self._give_back(row, j)
        self.block_table[b].copy_(torch.tensor(row, dtype=torch.int32))


class PagedKVCache(_PagePool):
    """Caller-owned device buffers of a paged cache (oscar_paged_cache):
    a pool of n_pages pages (each one 2752-byte record per KV head for 32
    tokens), the block table [B][max_blocks] (page ids, -1 = unmapped),
    per-sequence lengths n_packed[B], n_res[B] on the device, and the
    per-(b, h) residual windows.  Pages are handed out by the host-side
    allocator below; the device kernels only follow the table."""

    def __init__(self, B: int, Hkv: int, max_blocks: int, n_pages: int, flags: int = 0,
                 device=None, norm_target: float = 0.0, key_group: int = 0, bits: int = 0):
        dev = torch.device(device if device is not None else "cuda")
        self.pages = torch.zeros((n_pages, Hkv, record_bytes(bits)), dtype=torch.uint8,
                                 device=dev)
        self.block_table = torch.full((B, max_blocks), -1, dtype=torch.int32, device=dev)
        self.n_packed_d = torch.zeros(B, dtype=torch.int32, device=dev)
        self.n_res_d = torch.zeros(B, dtype=torch.int32, device=dev)
        self.k_res = torch.zeros((B, Hkv, R, D), dtype=torch.bfloat16, device=dev)
        self.v_res = torch.zeros((B, Hkv, R, D), dtype=torch.bfloat16, device=dev)
        self.k_res_norm = torch.zeros((B, Hkv, R), dtype=torch.float16, device=dev)
        s = OscarPagedCacheStruct()
        s.B, s.Hkv, s.max_blocks, s.n_pages, s.flags = B, Hkv, max_blocks, n_pages, flags
        s.norm_target = norm_target
        s.key_group = key_group
        s.bits = bits
        s.pages = self.pages.data_ptr()
        s.block_table = self.block_table.data_ptr()
        s.n_packed = self.n_packed_d.data_ptr()
        s.n_res = self.n_res_d.data_ptr()
        for name in ("k_res", "v_res", "k_res_norm"):
            setattr(s, name, getattr(self, name).data_ptr())
        self.struct = s
        self._init_pool(B, max_blocks, n_pages)

    B = property(lambda self: self.struct.B)
    Hkv = property(lambda self: self.struct.Hkv)
    max_blocks = property(lambda self: self.struct.max_blocks)
    n_pages = property(lambda self: self.struct.n_pages)
    flags = property(lambda self: self.struct.flags)

    def ref(self):
        return ctypes.byref(self.struct)

    def record(self, b: int, h: int, block: int) -> torch.Tensor:
        """View of the 2752-byte record of (b, h, logical block)."""
        return self.pages[self.page_of(b, block), h]

    def lengths(self):
        """(n_packed, n_res) per sequence, read back from the device."""
        return self.n_packed_d.cpu().tolist(), self.n_res_d.cpu().tolist()


class KV16Cache:
    """A 16-bit cache (oscar_kv16_cache) over the caller's device tensors:

    k, v         bf16 or fp16; paged [n_pages][Hkv][32][128] if block_table is
                 given, else contiguous [B][Hkv][T_cap][128]
    n_tok        int32 [B], the sequences' lengths
    block_table  int32 [B][max_blocks], page ids
    weight       optional float32, as k without its last dimension
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, n_tok: torch.Tensor,
                 block_table: torch.Tensor | None = None, weight: torch.Tensor | None = None):
        self.k, self.v, self.n_tok = k, v, n_tok
        self.block_table, self.weight = block_table, weight
        if k.dtype not in _KV16_DTYPES:
            raise ValueError("the cache takes bfloat16 or float16 keys and values")
        if k.dim() != 4 or k.shape[3] != D or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v: two tensors [..][Hkv][..][128] of one shape and type")
        if block_table is not None and (block_table.dim() != 2 or k.shape[2] != G):
            raise ValueError("a paged cache: block_table [B][max_blocks], k [n_pages][Hkv][32][128]")
        if weight is not None and weight.shape != k.shape[:3]:
            raise ValueError("weight: the shape of k without its last dimension")
        self.B = int(k.shape[0] if block_table is None else block_table.shape[0])
        self.Hkv, self.dtype, self.device = int(k.shape[1]), k.dtype, k.device
        self._index = k.get_device()
        s = OscarKV16CacheStruct()
        s.B, s.Hkv, s.dtype = self.B, self.Hkv, _KV16_DTYPES[k.dtype]
        if block_table is None:
            s.T_cap = k.shape[2]
        else:
            s.max_blocks, s.n_pages = block_table.shape[1], k.shape[0]
        s.k, s.v = _ptr(k), self._mine(v, k.dtype, k.numel())
        s.n_tok = self._mine(n_tok, torch.int32, self.B)
        s.block_table = self._mine(block_table, torch.int32, None)
        s.weight = self._mine(weight, torch.float32, k.numel() // D)
        self.struct = s
        self._ref = ctypes.byref(s)

    # A decode step is a handful of microseconds on the GPU, so the checks below
    # use the cheapest accessors (an int device index, identity of dtypes).

    def _mine(self, t: torch.Tensor | None, dtype: torch.dtype, n: int | None):
        """Pointer of a dense tensor that goes with the cache."""
        if t is None:
            return None
        if t.dtype is not dtype or (n is not None and t.numel() != n):
            raise ValueError(f"expected {n if n is not None else ''} {dtype} elements, "
                             f"got {tuple(t.shape)} {t.dtype}")
        if t.get_device() != self._index or not t.is_contiguous():
            raise ValueError(f"expected a dense tensor on {self.device}, got one on {t.device}")
        return t.data_ptr()

    def _rows(self, t: torch.Tensor, heads: int | None, total: int | None = None):
        """(pointer, row stride, rows, heads) of a [rows][heads][128] tensor of the
        cache's type, dense within a row."""
        shape = t.shape
        if len(shape) != 3 or shape[2] != D or t.dtype is not self.dtype or \
                (heads is not None and shape[1] != heads) or \
                (total is not None and shape[0] != total):
            raise ValueError(f"expected [{total if total is not None else 'rows'}]"
                             f"[{heads if heads is not None else 'heads'}][{D}] of {self.dtype}, "
                             f"got {tuple(shape)} {t.dtype}")
        if t.get_device() != self._index:
            raise ValueError(f"tensor on {t.device}, cache on {self.device}")
        rows, heads, _ = shape
        row, head, one = t.stride()
        if one != 1 or (heads > 1 and head != D):
            raise ValueError("a row's heads have to lie densely one behind another")
        return t.data_ptr(), (row if rows > 1 else heads * D), rows, heads

    def ref(self):
        return self._ref

    capacity = property(lambda self: self.struct.max_blocks * G if self.block_table is not None
                        else self.struct.T_cap)

    @staticmethod
    def contiguous(B: int, Hkv: int, T_cap: int, dtype=torch.bfloat16, device=None,
                   weights: bool = False) -> "KV16Cache":
        """An empty contiguous cache with buffers of its own."""
        dev = torch.device(device if device is not None else "cuda")
        k, v = (torch.zeros((B, Hkv, T_cap, D), dtype=dtype, device=dev) for _ in range(2))
        w = torch.zeros((B, Hkv, T_cap), dtype=torch.float32, device=dev) if weights else None
        return KV16Cache(k, v, torch.zeros(B, dtype=torch.int32, device=dev), weight=w)


class PagedKV16Cache(_PagePool, KV16Cache):
    """A paged KV16Cache with buffers and a block table of its own; pages are
    handed out as in PagedKVCache."""

    def __init__(self, B: int, Hkv: int, max_blocks: int, n_pages: int, dtype=torch.bfloat16,
                 device=None, weights: bool = False):
        dev = torch.device(device if device is not None else "cuda")
        k, v = (torch.zeros((n_pages, Hkv, G, D), dtype=dtype, device=dev) for _ in range(2))
        w = torch.zeros((n_pages, Hkv, G), dtype=torch.float32, device=dev) if weights else None
        KV16Cache.__init__(self, k, v, torch.zeros(B, dtype=torch.int32, device=dev),
                           torch.full((B, max_blocks), -1, dtype=torch.int32, device=dev), w)
        self._init_pool(B, max_blocks, n_pages)


# ---------------------------------------------------------------------------
# the calls (same names as the C ABI, without the oscar_ prefix)
# ---------------------------------------------------------------------------

def rotate_q(q: torch.Tensor, q_rot: torch.Tensor, flags: int = 0, stream=None):
    B, Hq = q.shape[0], q.shape[1]
    _check(_lib.oscar_rotate_q(_ptr(q), _ptr(q_rot), B, Hq, flags, _stream(stream)),
           "oscar_rotate_q")


def rotate_scale_k(k: torch.Tensor, k_hat: torch.Tensor, norm: torch.Tensor, B: int, Hkv: int,
                   n_tok: int, in_T: int, out_T: int, out_t0: int = 0, flags: int = 0,
                   stream=None, norm_target: float = 0.0):
    _check(_lib.oscar_rotate_scale_k(_ptr(k), in_T, _ptr(k_hat), _ptr(norm), out_T, out_t0,
                                     B, Hkv, n_tok, flags, norm_target, _stream(stream)),
           "oscar_rotate_scale_k")


def prefill_kv(cache: KVCache, k: torch.Tensor, v: torch.Tensor, n_tok: int, in_T: int = 0,
               stream=None):
    """Fused rotate + scale + quantise of tokens [0, n_tok) of raw bf16 keys
    and values [B][Hkv][in_T][128] into the packed cache (advances n_packed)."""
    in_T = in_T or k.shape[2]
    _check(_lib.oscar_prefill_kv(cache.ref(), _ptr(k), _ptr(v), in_T, n_tok, _stream(stream)),
           "oscar_prefill_kv")


def paged_prefill_kv(cache: PagedKVCache, k: torch.Tensor, v: torch.Tensor,
                     n_tok: torch.Tensor, max_tok: int, in_T: int = 0, stream=None):
    """Fused prefill of sequence b's tokens [0, n_tok[b]) (device int32 [B],
    multiples of 32, <= max_tok) into its next logical blocks."""
    in_T = in_T or k.shape[2]
    _check(_lib.oscar_paged_prefill_kv(cache.ref(), _ptr(k), _ptr(v), in_T, _ptr(n_tok),
                                       max_tok, _stream(stream)), "oscar_paged_prefill_kv")


def paged_append_kv(cache: PagedKVCache, k_new: torch.Tensor, v_new: torch.Tensor,
                    active: torch.Tensor | None = None, stream=None):
    """One new token [B][Hkv][128] for every sequence with active[b] != 0."""
    _check(_lib.oscar_paged_append_kv(cache.ref(), _ptr(k_new), _ptr(v_new), _ptr(active),
                                      _stream(stream)), "oscar_paged_append_kv")


def paged_decode_attention(cache: PagedKVCache, q_rot: torch.Tensor, Hq: int,
                           softmax_scale: float, max_packed: int, out: torch.Tensor,
                           workspace: torch.Tensor, num_splits: int = 0, stream=None):
    _check(_lib.oscar_paged_decode_attention(cache.ref(), _ptr(q_rot), Hq, softmax_scale,
                                             max_packed, _ptr(out), num_splits, _ptr(workspace),
                                             workspace.numel() * workspace.element_size(),
                                             _stream(stream)), "oscar_paged_decode_attention")


def quantize_kv(cache: KVCache, k_hat=None, k_norm=None, v=None, src_T: int = 0,
                n_tok: int = 0, stream=None):
    _check(_lib.oscar_quantize_kv(cache.ref(), _ptr(k_hat), _ptr(k_norm), _ptr(v), src_T, n_tok,
                                  _stream(stream)), "oscar_quantize_kv")


def append_kv(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, n_tok: int = 1,
              stream=None):
    _check(_lib.oscar_append_kv(cache.ref(), _ptr(k_new), _ptr(v_new), n_tok, _stream(stream)),
           "oscar_append_kv")


def decode_num_splits(B: int, Hkv: int, Hq: int, n_packed: int) -> int:
    return int(_lib.oscar_decode_num_splits(B, Hkv, Hq, n_packed))


def decode_plan_splits(rows: int, n_blocks: int, ctas_per_sm: int, sms: int) -> int:
    return int(_lib.oscar_decode_plan_splits(rows, n_blocks, ctas_per_sm, sms))


def decode_workspace_bytes(B: int, Hkv: int, Hq: int, n_packed: int, num_splits: int = 0) -> int:
    return int(_lib.oscar_decode_workspace_bytes(B, Hkv, Hq, n_packed, num_splits))


def alloc_workspace(nbytes: int, device=None) -> torch.Tensor:
    """A decode workspace of at least nbytes, zeroed: its header of row
    counters must start at zero, and every decode call leaves it zero."""
    return torch.zeros(max(16, (nbytes + 15) // 16 * 16) // 4, dtype=torch.float32,
                       device=device if device is not None else "cuda")


def decode_attention(cache: KVCache, q_rot: torch.Tensor, Hq: int, softmax_scale: float,
                     out: torch.Tensor, workspace: torch.Tensor, num_splits: int = 0,
                     stream=None):
    _check(_lib.oscar_decode_attention(cache.ref(), _ptr(q_rot), Hq, softmax_scale, _ptr(out),
                                       num_splits, _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       _stream(stream)), "oscar_decode_attention")


def decode_step(cache: KVCache, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                Hq: int, softmax_scale: float, out: torch.Tensor, workspace: torch.Tensor,
                num_splits: int = 0, stream=None):
    """One decode step in one launch: rotate the raw queries q (bf16
    [B][Hq][128]), append the new token (k_new, v_new bf16 [B][Hkv][128];
    a full window is flushed first) and attend; equals rotate_q + append_kv +
    decode_attention bit for bit.  Advances the cache's residual count."""
    _check(_lib.oscar_decode_step(cache.ref(), _ptr(q), _ptr(k_new), _ptr(v_new), Hq,
                                  softmax_scale, _ptr(out), num_splits, _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)),
           "oscar_decode_step")


def decode_attention_static_ws(cache: KVCache, q_rot: torch.Tensor, Hq: int,
                               softmax_scale: float, out: torch.Tensor, num_splits: int = 0,
                               stream=None):
    """decode_attention for callers that cannot allocate: the split-K partials
    use the library's own static device array (no workspace argument)."""
    _check(_lib.oscar_decode_attention_static_ws(cache.ref(), _ptr(q_rot), Hq, softmax_scale,
                                                 _ptr(out), num_splits, _stream(stream)),
           "oscar_decode_attention_static_ws")


def bf16_decode_attention(q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, B: int, Hq: int,
                          Hkv: int, T: int, T_stride: int, softmax_scale: float,
                          out: torch.Tensor, workspace: torch.Tensor, num_splits: int = 0,
                          stream=None):
    _check(_lib.oscar_bf16_decode_attention(_ptr(q), _ptr(K), _ptr(V), B, Hq, Hkv, T, T_stride,
                                            softmax_scale, _ptr(out), num_splits,
                                            _ptr(workspace),
                                            workspace.numel() * workspace.element_size(),
                                            _stream(stream)), "oscar_bf16_decode_attention")


# ---- the 16-bit cache ------------------------------------------------------

def _on_device(cache: KV16Cache, fn, args):
    """Calls the library with the cache's device current."""
    if torch._C._cuda_getDevice() == cache._index:
        return fn(*args)
    with torch.cuda.device(cache.device):
        return fn(*args)


def _kv16_call(cache: KV16Cache, where: str, fn, args, stream):
    """Calls the library with the cache's device current, on `stream` or that
    device's current stream."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(cache._index)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    st = _on_device(cache, fn, (*args, raw))
    if st != 0:
        raise OscarError(st, where)


def _bytes(workspace: torch.Tensor, cache: KV16Cache):
    if workspace.get_device() != cache._index or not workspace.is_contiguous():
        raise ValueError(f"expected a dense workspace on {cache.device}")
    return workspace.data_ptr(), workspace.nbytes


def kv16_write(cache: KV16Cache, k_new: torch.Tensor, v_new: torch.Tensor, start: torch.Tensor,
               pos0: torch.Tensor, stream=None):
    """New tokens into the cache: rows start[b] .. start[b+1] of k_new, v_new
    [total][Hkv][128] (a row may be a slice of a wider one) go to sequence b's
    positions pos0[b] .., and n_tok[b] = pos0[b] + their number."""
    k, ks, total, _ = cache._rows(k_new, cache.Hkv)
    v, vs, _, _ = cache._rows(v_new, cache.Hkv, total)
    _kv16_call(cache, "oscar_kv16_write", _lib.oscar_kv16_write,
               (cache._ref, k, ks, v, vs, cache._mine(start, torch.int32, cache.B + 1),
                cache._mine(pos0, torch.int32, cache.B), total), stream)


def kv16_attention_workspace_bytes(cache: KV16Cache, Hq: int, total: int, max_tok: int,
                                   window: int = 0, n_sink: int = 0) -> int:
    return int(_on_device(cache, _lib.oscar_kv16_attention_workspace_bytes,
                          (cache._ref, Hq, total, max_tok, window, n_sink)))


def kv16_attention(cache: KV16Cache, q: torch.Tensor, start: torch.Tensor, softmax_scale: float,
                   max_tok: int, out: torch.Tensor, workspace: torch.Tensor, window: int = 0,
                   n_sink: int = 0, lse: torch.Tensor | None = None, stream=None):
    """Causal attention of every sequence's newest tokens over its cached ones:
    rows start[b] .. start[b+1] of q [total][Hq][128] are the queries of the
    last tokens of sequence b (already in the cache).  With window > 0 a query
    sees the last `window` tokens up to its own and the first n_sink.  out
    [total][Hq][128]; lse float32 [total][Hq]: the logarithm of the sum of the
    exponentials.  max_tok bounds the n_tok[b]."""
    qp, qs, total, Hq = cache._rows(q, None)
    w, wb = _bytes(workspace, cache)
    _kv16_call(cache, "oscar_kv16_attention", _lib.oscar_kv16_attention,
               (cache._ref, qp, qs, cache._mine(start, torch.int32, cache.B + 1), total, Hq,
                softmax_scale, max_tok, window, n_sink,
                cache._mine(out, cache.dtype, total * Hq * D),
                cache._mine(lse, torch.float32, total * Hq), w, wb), stream)


def kv16_decode_workspace_bytes(cache: KV16Cache, Hq: int, max_tok: int, window: int = 0,
                                n_sink: int = 0, accumulate: bool = False) -> int:
    return int(_on_device(cache, _lib.oscar_kv16_decode_workspace_bytes,
                          (cache._ref, Hq, max_tok, window, n_sink, int(accumulate))))


def kv16_decode_attention(cache: KV16Cache, q: torch.Tensor, softmax_scale: float, max_tok: int,
                          out: torch.Tensor, workspace: torch.Tensor, window: int = 0,
                          n_sink: int = 0, accumulate: bool = False, stream=None):
    """Attention of each sequence's newest token, q and out [B][Hq][128];
    accumulate adds its probabilities to the weights of the tokens it sees.
    The workspace comes zeroed from alloc_workspace."""
    qp, qs, _, Hq = cache._rows(q, None, cache.B)
    w, wb = _bytes(workspace, cache)
    _kv16_call(cache, "oscar_kv16_decode_attention", _lib.oscar_kv16_decode_attention,
               (cache._ref, qp, qs, Hq, softmax_scale, max_tok, window, n_sink, int(accumulate),
                cache._mine(out, cache.dtype, cache.B * Hq * D), w, wb), stream)


def kv16_accumulate(cache: KV16Cache, q: torch.Tensor, lse: torch.Tensor, start: torch.Tensor,
                    softmax_scale: float, max_tok: int, window: int = 0, n_sink: int = 0,
                    n_obs: int = 0, stream=None):
    """Adds to each cached token's weight the probabilities it got from the
    last n_obs queries (0: all) of its sequence; q, start and the window as for
    kv16_attention, lse as it wrote it."""
    qp, qs, total, Hq = cache._rows(q, None)
    _kv16_call(cache, "oscar_kv16_accumulate", _lib.oscar_kv16_accumulate,
               (cache._ref, qp, qs, cache._mine(lse, torch.float32, total * Hq),
                cache._mine(start, torch.int32, cache.B + 1), total, Hq, softmax_scale, max_tok,
                window, n_sink, n_obs), stream)


def kv16_evict_workspace_bytes(src: KV16Cache, max_tok: int, keep_first: int, keep_recent: int,
                               keep_top: int) -> int:
    return int(_on_device(src, _lib.oscar_kv16_evict_workspace_bytes,
                          (src._ref, max_tok, keep_first, keep_recent, keep_top)))


def kv16_evict(src: KV16Cache, dst: KV16Cache, max_tok: int, keep_first: int, keep_recent: int,
               keep_top: int, workspace: torch.Tensor, kept: torch.Tensor | None = None,
               stream=None):
    """The first keep_first, the last keep_recent and the keep_top heaviest
    tokens between them, per (sequence, KV head), into dst in order of
    position.  kept int32 [B][Hkv][keep]: their positions in src, -1 behind the
    last.  Sequences of at most keep tokens are copied whole."""
    if dst.device != src.device:
        raise ValueError(f"source on {src.device}, destination on {dst.device}")
    keep = keep_first + keep_recent + keep_top
    w, wb = _bytes(workspace, src)
    _kv16_call(src, "oscar_kv16_evict", _lib.oscar_kv16_evict,
               (src._ref, dst._ref, max_tok, keep_first, keep_recent, keep_top,
                src._mine(kept, torch.int32, src.B * src.Hkv * keep), w, wb), stream)


# ---- sequences with tokens in common ---------------------------------------

def kv16_shared_decode_workspace_bytes(cache: KV16Cache, Hq: int, n_groups: int, max_tok: int,
                                       window: int = 0, n_sink: int = 0) -> int:
    return int(_on_device(cache, _lib.oscar_kv16_shared_decode_workspace_bytes,
                          (cache._ref, Hq, n_groups, max_tok, window, n_sink)))


def kv16_shared_decode_attention(cache: KV16Cache, q: torch.Tensor, group: torch.Tensor,
                                 prefix: torch.Tensor, softmax_scale: float, max_tok: int,
                                 out: torch.Tensor, workspace: torch.Tensor, window: int = 0,
                                 n_sink: int = 0, stream=None):
    """kv16_decode_attention of sequences that share prefixes: sequences group[i]
    .. group[i+1] - 1 have their first prefix[i] tokens in common, whose whole
    pages are read once for all of them, from the first one's place in the cache
    (which has to keep them: release_blocks takes them from all).  group int32
    [n + 1], prefix int32 [n].  A max_tok near the lengths lets small batches of
    short sequences go the quicker way; it keeps more bits of the probabilities too,
    as kv16_decode_attention does."""
    qp, qs, _, Hq = cache._rows(q, None, cache.B)
    w, wb = _bytes(workspace, cache)
    n = prefix.numel()
    _kv16_call(cache, "oscar_kv16_shared_decode_attention", _lib.oscar_kv16_shared_decode_attention,
               (cache._ref, qp, qs, Hq, cache._mine(group, torch.int32, n + 1),
                cache._mine(prefix, torch.int32, n), n, softmax_scale, max_tok, window, n_sink,
                cache._mine(out, cache.dtype, cache.B * Hq * D), w, wb), stream)


def kv16_shared_attention_workspace_bytes(cache: KV16Cache, Hq: int, n_groups: int, total: int,
                                          max_tok: int, window: int = 0, n_sink: int = 0) -> int:
    return int(_on_device(cache, _lib.oscar_kv16_shared_attention_workspace_bytes,
                          (cache._ref, Hq, n_groups, total, max_tok, window, n_sink)))


def kv16_shared_attention(cache: KV16Cache, q: torch.Tensor, start: torch.Tensor,
                          group: torch.Tensor, prefix: torch.Tensor, softmax_scale: float,
                          max_tok: int, out: torch.Tensor, workspace: torch.Tensor,
                          window: int = 0, n_sink: int = 0, lse: torch.Tensor | None = None,
                          stream=None):
    """kv16_attention of sequences that share prefixes (groups as for
    kv16_shared_decode_attention)."""
    qp, qs, total, Hq = cache._rows(q, None)
    w, wb = _bytes(workspace, cache)
    n = prefix.numel()
    _kv16_call(cache, "oscar_kv16_shared_attention", _lib.oscar_kv16_shared_attention,
               (cache._ref, qp, qs, cache._mine(start, torch.int32, cache.B + 1), total, Hq,
                cache._mine(group, torch.int32, n + 1), cache._mine(prefix, torch.int32, n), n,
                softmax_scale, max_tok, window, n_sink,
                cache._mine(out, cache.dtype, total * Hq * D),
                cache._mine(lse, torch.float32, total * Hq), w, wb), stream)


def kv16_fork(src: KV16Cache, dst: KV16Cache, parent: torch.Tensor, max_tok: int,
              share: bool = True, stream=None):
    """Sequence b of dst becomes a copy of sequence parent[b] of src (int32
    [dst.B]; negative: stays as it is).  share: its whole pages are the parent's
    own (dst's table is written), the tokens behind them are copied; else every
    token is copied, to the places that dst's table names, which are to be pages of
    the sequence's own (release_blocks and map_blocks give those again).  max_tok
    bounds the parents' lengths.

    share and a dst with an allocator (PagedKV16Cache): the pages that dst's
    sequences had in those places are given back and the parent's are counted, by
    the next call of the allocator, which waits for the device.  After a fork that
    was captured into a graph every such call waits.  Where src is not dst, src's
    allocator does not know of dst's tables.

    Sequences that continue one another (a step of a beam search) are forked from a
    KV16Cache over the same k and v with copies of n_tok and block_table, once every
    sequence of dst has given its last page back and then got one that was free before
    (release_blocks of all, then map_blocks, in a pool with so many pages free)."""
    if dst.device != src.device:
        raise ValueError(f"source on {src.device}, destination on {dst.device}")
    _kv16_call(src, "oscar_kv16_fork", _lib.oscar_kv16_fork,
               (src._ref, dst._ref, dst._mine(parent, torch.int32, dst.B), int(share), max_tok),
               stream)
    if share and isinstance(dst, _PagePool):
        dst._table_written(stream)


def page_compact_workspace_bytes(block_table: torch.Tensor, n_pages: int) -> int:
    B, max_blocks = block_table.shape
    return int(_lib.oscar_page_compact_workspace_bytes(B, max_blocks, n_pages))


def page_compact(block_table: torch.Tensor, new_table: torch.Tensor, n_pages: int,
                 moves: torch.Tensor, counts: torch.Tensor, workspace: torch.Tensor, stream=None):
    """Plans the compaction of a pool of n_pages pages: the pages that
    block_table [B][max_blocks] names get the ids 0 .. L - 1.  new_table: the
    table with the new ids (may be block_table itself); moves int32
    [n_pages // 2][2]: the pages to copy, old and new id, for kv16_copy_pages;
    counts int32 [2]: the number of moves, L."""
    index, i32 = block_table.get_device(), torch.int32
    for t in (block_table, new_table, moves, counts, workspace):
        if t.get_device() != index or index < 0 or not t.is_contiguous() or \
                (t.dtype is not i32 and t is not workspace):
            raise ValueError("expected dense int32 tensors on one GPU, and a workspace there")
    if block_table.dim() != 2 or new_table.shape != block_table.shape or \
            moves.numel() != n_pages // 2 * 2 or counts.numel() != 2:
        raise ValueError("expected tables [B][max_blocks], moves [n_pages // 2][2], counts [2]")
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
    B, max_blocks = block_table.shape
    args = (block_table.data_ptr(), new_table.data_ptr(), B, max_blocks, n_pages, moves.data_ptr(),
            counts.data_ptr(), workspace.data_ptr(), workspace.nbytes, raw)
    if torch._C._cuda_getDevice() == index:
        _check(_lib.oscar_page_compact(*args), "oscar_page_compact")
    else:
        with torch.cuda.device(index):
            _check(_lib.oscar_page_compact(*args), "oscar_page_compact")


def paged_copy_pages(cache: PagedKVCache, pairs: torch.Tensor, n_pairs: torch.Tensor, stream=None):
    """Pages pairs[i][0] of a packed cache's pool to pages pairs[i][1], int32
    [..][2], for i below the first element of n_pairs (int32)."""
    if pairs.dim() != 2 or pairs.shape[1] != 2 or n_pairs.numel() < 1 or \
            any(t.dtype is not torch.int32 or t.device != cache.pages.device for t in (pairs, n_pairs)):
        raise ValueError(f"expected int32 pairs [..][2] and their number on {cache.pages.device}")
    with torch.cuda.device(cache.pages.device):
        _check(_lib.oscar_paged_copy_pages(cache.ref(), _ptr(pairs), _ptr(n_pairs), pairs.shape[0],
                                           _stream(stream)), "oscar_paged_copy_pages")


def kv16_copy_pages(src: KV16Cache, dst: KV16Cache, pairs: torch.Tensor, n_pairs: torch.Tensor,
                    stream=None):
    """Pages pairs[i][0] of src to pages pairs[i][1] of dst (which may be one
    pool), int32 [..][2], for i below the first element of n_pairs (int32)."""
    if dst.device != src.device:
        raise ValueError(f"source on {src.device}, destination on {dst.device}")
    if n_pairs.numel() < 1 or pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("expected pairs [..][2] and their number")
    _kv16_call(src, "oscar_kv16_copy_pages", _lib.oscar_kv16_copy_pages,
               (src._ref, dst._ref, src._mine(pairs, torch.int32, None),
                src._mine(n_pairs, torch.int32, None), pairs.shape[0]), stream)


def selftest_wait_timeout(iterations: int = 256, stream=None):
    """Launches the bounded-wait self-test: a wait that can never complete
    gives up after `iterations` polls and sets the device status word."""
    _check(_lib.oscar_selftest_wait_timeout(iterations, _stream(stream)),
           "oscar_selftest_wait_timeout")


def selftest_tc_wait_timeout(report: torch.Tensor, iterations: int = 256, stream=None):
    """The same of the tensor-core kernels' waits; report (int32 [3]): a wait gave
    up, another warp's followed it, one did while a warp was busy (1, 1, 0)."""
    if report.dtype is not torch.int32 or report.numel() != 3:
        raise ValueError("report: int32 [3]")
    _check(_lib.oscar_selftest_tc_wait_timeout(iterations, _ptr(report), _stream(stream)),
           "oscar_selftest_tc_wait_timeout")


def selftest_kv16_decode_timeout(cache: KV16Cache, q: torch.Tensor, max_tok: int,
                                 out: torch.Tensor, workspace: torch.Tensor, stream=None):
    """kv16_decode_attention (dense q, no window) in which every wait for a copy
    gives up at once: the status word reports it, the workspace stays usable."""
    qp, _, _, Hq = cache._rows(q, None, cache.B)
    if not q.is_contiguous():
        raise ValueError("expected dense queries")
    w, wb = _bytes(workspace, cache)
    _kv16_call(cache, "oscar_selftest_kv16_decode_timeout", _lib.oscar_selftest_kv16_decode_timeout,
               (cache._ref, qp, Hq, max_tok, cache._mine(out, cache.dtype, cache.B * Hq * D), w, wb),
               stream)


def selftest_kv16_shared_timeout(cache: KV16Cache, q: torch.Tensor, group: torch.Tensor,
                                 prefix: torch.Tensor, max_tok: int, out: torch.Tensor,
                                 workspace: torch.Tensor, items: int = 0, stream=None):
    """kv16_shared_decode_attention (dense q, no window) whose copies end early: what
    waits for them gives up (at once where a row is one block's, else after two
    seconds, behind `items` pieces of work), the status word reports it."""
    qp, _, _, Hq = cache._rows(q, None, cache.B)
    if not q.is_contiguous():
        raise ValueError("expected dense queries")
    w, wb = _bytes(workspace, cache)
    n = prefix.numel()
    _kv16_call(cache, "oscar_selftest_kv16_shared_timeout", _lib.oscar_selftest_kv16_shared_timeout,
               (cache._ref, qp, Hq, cache._mine(group, torch.int32, n + 1),
                cache._mine(prefix, torch.int32, n), n, max_tok, items,
                cache._mine(out, cache.dtype, cache.B * Hq * D), w, wb), stream)


def device_status(stream=None) -> int:
    return int(_lib.oscar_device_status(_stream(stream)))


def kernel_launches() -> int:
    return int(_lib.oscar_kernel_launches())


def default_scale() -> float:
    return 1.0 / math.sqrt(D)
