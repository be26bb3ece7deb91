"""Python binding of the 8-bit paged KV cache, include/kv8.h (ctypes).

Argument marshalling only, as in kvq.py: torch tensors serve as device memory
and torch streams as CUDA streams.
"""

from __future__ import annotations

import ctypes
import struct
from ctypes import c_float, c_int32, c_int64, c_size_t, c_void_p

import torch

from .kvq import KVQ_OK, KvqError, lib

FORMATS = {"int8": 0, "e4m3": 1}
DTYPES = {torch.float16: 0, torch.bfloat16: 1}
CODE_DTYPES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
BUF_CODES, BUF_SCALES, BUF_K_WIN, BUF_V_WIN, BUF_SEQ_LEN, BUF_BLOCK_TABLE = range(6)

EXPORTED = ("kv8_max_blocks", "kv8_buffer_bytes", "kv8_append", "kv8_attn_workspace_bytes", "kv8_attn")


class CacheStruct(ctypes.Structure):
    """Mirror of `kv8_cache` (include/kv8.h)."""
    _fields_ = [
        ("num_seqs", c_int32), ("num_kv_heads", c_int32), ("head_dim", c_int32), ("block", c_int32),
        ("format", c_int32), ("dtype", c_int32), ("capacity", c_int32), ("num_blocks", c_int32),
        ("codes", c_void_p), ("scales", c_void_p), ("k_win", c_void_p), ("v_win", c_void_p),
        ("seq_len", c_void_p), ("block_table", c_void_p), ("status", c_void_p),
    ]


class RowsStruct(ctypes.Structure):
    """Mirror of `kv8_rows` (include/kv8.h)."""
    _fields_ = [("data", c_void_p), ("row_stride", c_int64), ("head_stride", c_int64)]


# The same bytes, packed at a tenth of the cost of a ctypes structure: a call's
# host time is what a one-token step waits for.
_pack_rows = struct.Struct("@Pqq").pack
assert struct.calcsize("@Pqq") == ctypes.sizeof(RowsStruct)


_I32, _F32 = torch.int32, torch.float32
# what torch.cuda.current_stream and current_device ask, without their checks
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _sign():
    C, R = ctypes.POINTER(CacheStruct), c_void_p  # R: packed bytes, or a reference to a RowsStruct
    sig = {
        "kv8_max_blocks": (c_int32, [C]),
        "kv8_buffer_bytes": (c_int64, [C, c_int32]),
        "kv8_append": (ctypes.c_int, [C, R, R, R, R, c_int32, c_void_p, c_int32, c_int32, c_void_p, c_int32, c_int32,
                                      c_int32, c_void_p]),
        "kv8_attn_workspace_bytes": (c_int64, [C, c_int32, c_int32]),
        "kv8_attn": (ctypes.c_int, [C, c_int32, R, R, c_void_p, c_int32, c_int32, c_float, c_void_p, c_size_t,
                                    c_int32, c_void_p]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args


_sign()


class KV8Cache:
    """Device buffers of one 8-bit paged cache (one layer) and its descriptor.

    num_blocks: blocks of the pool; the caller assigns them to sequences in
    block_table [S][capacity // block] (int32, filled with -1) before the
    appends that complete them.  seq_len (int32 [S], zeros) counts the tokens
    of each sequence, those of the step in progress included; the caller
    advances it.  Buffers given as arguments are used as they are (another
    layer's seq_len and block_table, say), the others allocated.
    """

    def __init__(self, num_seqs, num_kv_heads, capacity, num_blocks, head_dim=128, block=64, fmt="int8",
                 dtype=torch.float16, device="cuda", codes=None, scales=None, k_win=None, v_win=None, seq_len=None,
                 block_table=None, status=None):
        if fmt not in FORMATS or dtype not in DTYPES:
            raise ValueError(f"format {fmt!r} or dtype {dtype} not supported")
        st = CacheStruct(num_seqs, num_kv_heads, head_dim, block, FORMATS[fmt], DTYPES[dtype], capacity, num_blocks)
        self.max_blocks = lib.kv8_max_blocks(ctypes.byref(st))
        if self.max_blocks < 0:
            raise KvqError(-2, "kv8_max_blocks")
        self.num_seqs, self.num_kv_heads, self.head_dim, self.block = num_seqs, num_kv_heads, head_dim, block
        self.capacity, self.num_blocks, self.fmt, self.dtype = capacity, num_blocks, fmt, dtype
        if codes is not None:
            device = codes.device
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        S, H, B, D = num_seqs, num_kv_heads, block, head_dim

        def buffer(name, given, shape, dt, fill=0):
            if given is None:
                n = 1
                for x in shape:
                    n *= x
                # an empty buffer still has an address
                t = torch.full((max(n, 1),), fill, dtype=torch.uint8 if dt in CODE_DTYPES.values() else dt,
                               device=self.device)
                return (t.view(dt) if t.dtype != dt else t)[:n].view(shape)
            if tuple(given.shape) != shape or given.dtype != dt or not given.is_contiguous() \
                    or given.device != self.device:
                raise ValueError(f"{name}: a contiguous {dt} tensor of shape {shape} on {self.device} is needed")
            return given

        self.codes = buffer("codes", codes, (num_blocks, H, 2, B, D), CODE_DTYPES[fmt])
        self.scales = buffer("scales", scales, (num_blocks, H, 2), torch.float32)
        self.k_win = buffer("k_win", k_win, (S, H, B, D), dtype)
        self.v_win = buffer("v_win", v_win, (S, H, B, D), dtype)
        self.seq_len = buffer("seq_len", seq_len, (S,), torch.int32)
        self.block_table = buffer("block_table", block_table, (S, self.max_blocks), torch.int32, -1)
        self.status = buffer("status", status, (1,), torch.int32)
        for name in ("codes", "scales", "k_win", "v_win", "seq_len", "block_table", "status"):
            setattr(st, name, getattr(self, name).data_ptr() or None)
        self.struct = st
        self.ref = ctypes.byref(st)
        self.device_index = self.codes.get_device()  # -1 on the CPU


def rope_table(rows: int, rot_dim: int, theta: float = 10000.0, device="cuda"):
    """The rope argument of kv8_append for plain rotary embeddings: row p has
    the cosines, then the sines, of p * theta^(-2 i / rot_dim), formed in 64
    bits and rounded to fp32."""
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
    ang = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * theta ** (-i / rot_dim)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _rows(t, cache, shape, name):
    """kv8_rows of a tensor of this shape, [rows][heads][D] (any row and head strides)."""
    if t.dtype is not cache.dtype or t.shape != shape or t.get_device() != cache.device_index:
        raise ValueError(f"{name}: a {cache.dtype} tensor of shape {tuple(shape)} on {cache.device} is needed")
    row, head, one = t.stride()
    if one != 1 and shape[0]:  # no rows: any strides
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return _pack_rows(t.data_ptr(), row, head)


def _row_start(row_start, cache):
    if row_start is None:
        return None
    if row_start.dtype is not _I32 or row_start.numel() != cache.num_seqs + 1 or not row_start.is_contiguous() \
            or row_start.get_device() != cache.device_index:
        raise ValueError(f"row_start: a contiguous int32 tensor [{cache.num_seqs + 1}] on {cache.device} is needed")
    return row_start.data_ptr()


def _launch(fn, what, cache, stream, *args):
    """fn(*args, stream) with the cache's device current."""
    index = cache.device_index
    if index < 0:
        raise ValueError("the cache is not on a CUDA device")
    raw = _current_stream(index) if stream is None else stream.cuda_stream
    if _current_device() == index:
        code = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            code = fn(*args, raw)
    if code != KVQ_OK:
        raise KvqError(code, what)


def kv8_append(cache: KV8Cache, k, v, row_start=None, max_new: int = 1, q=None, q_out=None, rope=None,
               interleaved: bool = False, stream=None):
    """k, v: [rows][Hkv][D]; q, q_out: [rows][Hq][D] (rotated along; q_out may
    be q); rope: fp32 [positions][rot_dim] (rope_table) or None.  row_start:
    int32 [S + 1], or None for one row per sequence."""
    rows, dim = k.shape[0] if k.shape else 0, cache.head_dim  # (len and size take longer than shape)
    shape = (rows, cache.num_kv_heads, dim)
    ks, vs = _rows(k, cache, shape, "k"), _rows(v, cache, shape, "v")
    qs = os = None
    heads = 0
    if q is not None:
        if q_out is None:
            raise ValueError("q without q_out")
        shape = q.shape
        heads = shape[1] if len(shape) == 3 else 0
        shape = (rows, heads, dim)
        qs, os = _rows(q, cache, shape, "q"), _rows(q_out, cache, shape, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    table, rot, positions = None, 0, 0
    if rope is not None:
        shape = rope.shape
        if rope.dtype is not _F32 or len(shape) != 2 or not rope.is_contiguous() \
                or rope.get_device() != cache.device_index:
            raise ValueError(f"rope: a contiguous float32 tensor [positions][rot_dim] on {cache.device} is needed")
        positions, rot = shape
        table = rope.data_ptr() if rot else None
    _launch(lib.kv8_append, "kv8_append", cache, stream, cache.ref, ks, vs, qs, os, heads,
            _row_start(row_start, cache), rows, max_new, table, positions, rot, 1 if interleaved else 0)


def attn_workspace_bytes(cache: KV8Cache, num_q_heads: int, max_new: int = 1) -> int:
    n = lib.kv8_attn_workspace_bytes(cache.ref, num_q_heads, max_new)
    if n < 0:
        raise KvqError(-1, "kv8_attn_workspace_bytes")
    return n


def alloc_workspace(cache: KV8Cache, num_q_heads: int, max_new: int = 1):
    """A torch-allocated, zero-filled workspace for kv8_attn."""
    return torch.zeros(attn_workspace_bytes(cache, num_q_heads, max_new), dtype=torch.uint8, device=cache.device)


def kv8_attn(cache: KV8Cache, q, out, workspace, max_len: int, row_start=None, max_new: int = 1,
             softmax_scale: float = 0.0, stream=None):
    """q, out: [rows][Hq][D] (out may be q); max_len: a bound on seq_len."""
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q: [rows][heads][D] is needed")
    rows, heads, _ = shape
    shape = (rows, heads, cache.head_dim)
    if workspace.get_device() != cache.device_index or not workspace.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on {cache.device} is needed")
    _launch(lib.kv8_attn, "kv8_attn", cache, stream, cache.ref, heads, _rows(q, cache, shape, "q"),
            _rows(out, cache, shape, "out"), _row_start(row_start, cache), rows, max_new, softmax_scale,
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), max_len)
