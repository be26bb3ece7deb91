"""The 8-bit paged cache without a GPU: the oracle's definitions against
closed forms and torch's own conversions, buffer sizes, and every refusal of
the C ABI (made before anything is launched)."""

import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import kv8 as ok

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kv8():
    from bit_kv_cache_02_gb300 import build
    build.build()
    from bit_kv_cache_02_gb300 import kv8 as mod
    return mod


# ------------------------------------------------------------------ oracle

def test_round16_matches_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.uniform(-44, 38, 20000),
                        [0.0, -0.0, 2.0 ** -133, 2.0 ** -134, 1.5 * 2.0 ** -133, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8]])
    x = x.astype(np.float32).astype(np.float64)
    for name in ("float16", "bfloat16"):
        want = torch.from_numpy(x.astype(np.float32)).to(getattr(torch, name)).double().numpy()
        np.testing.assert_array_equal(ok.round16(x, name), want)


def test_round_e4m3_matches_torch():
    x = np.random.default_rng(1).uniform(-448, 448, 20000).astype(np.float32)
    x = np.concatenate([x, x * np.float32(1e-3), np.float32([2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 17, 19, 448])])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(ok.round_e4m3(x), want)


def test_rotation_turns_by_the_angle():
    """In 64 bits the pair (a, b) is (a + ib) e^(i angle)."""
    rng = np.random.default_rng(2)
    x = ok.round16(rng.standard_normal((5, 2, 64)), "bfloat16")
    ang = rng.uniform(0, 6, (5, 16))
    tab = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32).astype(np.float64)
    for inter in (False, True):
        y = ok.rotate(x, tab, inter, "bfloat16")
        np.testing.assert_array_equal(y[..., 32:], x[..., 32:])
        i0 = np.arange(0, 32, 2) if inter else np.arange(16)
        i1 = i0 + 1 if inter else i0 + 16
        z = (x[..., i0] + 1j * x[..., i1]) * np.exp(1j * ang)[:, None]
        size = np.abs(x[..., i0]) + np.abs(x[..., i1])
        assert (np.abs(y[..., i0] - z.real) <= 2.0 ** -8 * np.abs(z.real) + 2.0 ** -21 * size).all()
        assert (np.abs(y[..., i1] - z.imag) <= 2.0 ** -8 * np.abs(z.imag) + 2.0 ** -21 * size).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_quantize_block_bounds(fmt):
    rng = np.random.default_rng(3)
    for amp in (1.0, 300.0, 2.0 ** -20):
        x = ok.round16(rng.standard_normal((32, 64)) * amp, "float16")
        c, scale = ok.quantize_block(x, fmt)
        amax = np.abs(x).max()
        if fmt == "int8":
            assert np.abs(c).max() == 127 and (np.abs(c * scale - x) <= (0.5 + 1e-4) * scale).all()
        else:
            assert 224 < amax / scale <= 448
            assert (np.abs(c * scale - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale)).all()
    c, scale = ok.quantize_block(np.zeros((32, 64)), fmt)
    assert (c == 0).all() and 0 < scale < 2.0 ** -99
    x[3, 4] = math.inf
    c, scale = ok.quantize_block(x, fmt)
    assert (c == 0).all() and math.isnan(scale)


def test_oracle_splits_and_attention():
    """Appending in pieces changes nothing; with every token in the window,
    attention is the textbook formula."""
    rng = np.random.default_rng(4)
    k, v = (ok.round16(rng.standard_normal((70, 2, 64)), "float16") for _ in range(2))
    tab = np.concatenate([np.cos(np.arange(70)[:, None] * [1.0] * 16), np.sin(np.arange(70)[:, None] * [1.0] * 16)], 1)
    a, b = (ok.OracleKV8(1, 2, 64, 32, "int8", "float16") for _ in range(2))
    a.append(k, v, [0, 70], tab)
    for lo, hi in ((0, 1), (1, 40), (40, 70)):
        b.append(k[lo:hi], v[lo:hi], [0, hi - lo], tab)
    np.testing.assert_array_equal(a.stored(0, 1, False), b.stored(0, 1, False))
    c = ok.OracleKV8(1, 2, 64, 128, "int8", "float16")
    c.append(k, v, [0, 70])
    q = rng.standard_normal((1, 4, 64))
    out, bound = c.attention(q, [0, 1])
    for j in range(4):
        w = np.exp(k[:, j // 2] @ q[0, j] / 8)
        np.testing.assert_allclose(out[0, j], w @ v[:, j // 2] / w.sum(), rtol=1e-12)
    assert (bound > 0).all()


# ----------------------------------------------------------------- binding

def test_exports_match_header(kv8):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kv8.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(kv8_[a-z_]+)\s*\(", text))
    assert names == set(kv8.EXPORTED)
    for n in names:
        assert hasattr(kv8.lib, n), n


def test_struct_layout(kv8):
    assert kv8.CacheStruct.codes.offset == 32 and ctypes.sizeof(kv8.CacheStruct) == 32 + 7 * 8
    assert ctypes.sizeof(kv8.RowsStruct) == 24


BASE = 1 << 30


def _struct(kv8, **kw):
    d = dict(num_seqs=3, num_kv_heads=2, head_dim=128, block=64, format=0, dtype=0, capacity=1000, num_blocks=40,
             codes=BASE, scales=BASE + (1 << 20), k_win=BASE + (1 << 21), v_win=BASE + (1 << 22),
             seq_len=BASE + (1 << 23), block_table=BASE + (1 << 24), status=0)
    d.update(kw)
    st = kv8.CacheStruct()
    for k, v in d.items():
        setattr(st, k, v or None if k in ("codes", "scales", "k_win", "v_win", "seq_len", "block_table", "status")
                else v)
    return st


def test_sizes(kv8):
    st = _struct(kv8)
    size = lambda w: kv8.lib.kv8_buffer_bytes(ctypes.byref(st), w)  # noqa: E731
    assert kv8.lib.kv8_max_blocks(ctypes.byref(st)) == 15
    assert size(kv8.BUF_CODES) == 40 * 2 * 2 * 64 * 128 and size(kv8.BUF_SCALES) == 40 * 2 * 2 * 4
    assert size(kv8.BUF_K_WIN) == size(kv8.BUF_V_WIN) == 3 * 2 * 64 * 128 * 2
    assert size(kv8.BUF_SEQ_LEN) == 12 and size(kv8.BUF_BLOCK_TABLE) == 3 * 15 * 4 and size(9) == -1
    n = kv8.lib.kv8_attn_workspace_bytes(ctypes.byref(st), 8, 1)
    assert n > 0 and n % 256 == 0
    assert kv8.lib.kv8_attn_workspace_bytes(ctypes.byref(st), 7, 1) == -1
    assert kv8.lib.kv8_attn_workspace_bytes(ctypes.byref(st), 8, 0) == -1
    assert kv8.lib.kv8_attn_workspace_bytes(ctypes.byref(st), 8, 1001) == -1


def _append(kv8, st, **kw):
    R = kv8.RowsStruct
    d = dict(k=R(BASE, 256, 128), v=R(BASE, 256, 128), q=R(BASE, 512, 128), q_out=R(BASE, 512, 128), heads=4,
             row_start=BASE, rows=10, max_new=10, rope=BASE, rope_rows=1000, rot=128, inter=0)
    d.update(kw)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return kv8.lib.kv8_append(ctypes.byref(st), ref(d["k"]), ref(d["v"]), ref(d["q"]), ref(d["q_out"]), d["heads"],
                              d["row_start"], d["rows"], d["max_new"], d["rope"], d["rope_rows"], d["rot"],
                              d["inter"], None)


def _attn(kv8, st, **kw):
    R = kv8.RowsStruct
    d = dict(heads=4, q=R(BASE, 512, 128), out=R(BASE, 512, 128), row_start=BASE, rows=10, max_new=10, ws=BASE,
             bytes=1 << 40, max_len=1000)
    d.update(kw)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return kv8.lib.kv8_attn(ctypes.byref(st), d["heads"], ref(d["q"]), ref(d["out"]), d["row_start"], d["rows"],
                            d["max_new"], 0.0, d["ws"], d["bytes"], d["max_len"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=0), -1), (dict(num_kv_heads=0), -1), (dict(capacity=0), -1), (dict(num_blocks=-1), -1),
    (dict(capacity=(1 << 30) + 1), -2),
    (dict(head_dim=96), -2), (dict(block=16), -2), (dict(block=100), -2), (dict(format=2), -2), (dict(dtype=2), -2),
    (dict(num_seqs=65536), -2), (dict(num_seqs=65535, num_kv_heads=65535), -2),
    (dict(codes=0), -1), (dict(scales=0), -1), (dict(k_win=0), -1), (dict(v_win=0), -1), (dict(seq_len=0), -1),
    (dict(block_table=0), -1), (dict(num_blocks=0), -1),
    (dict(codes=BASE + 8), -5), (dict(scales=BASE + 4), -5), (dict(k_win=BASE + 2), -5), (dict(v_win=BASE + 8), -5),
    (dict(seq_len=BASE + 1), -5), (dict(block_table=BASE + 2), -5), (dict(status=BASE + 2), -5),
])
def test_bad_cache_refused(kv8, kw, code):
    st = _struct(kv8, **kw)
    assert _append(kv8, st) == code and _attn(kv8, st) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(max_new=-1), -1), (dict(max_new=1001), -3), (dict(row_start=BASE + 2), -5),
    (dict(row_start=None, rows=2), -1),                    # fewer rows than sequences
    (dict(row_start=None, max_new=0), -1),
    (dict(k="null"), -1), (dict(v="null"), -1), (dict(q="null"), -1), (dict(q_out="null"), -1), (dict(heads=0), -1),
    (dict(heads=-4), -1), (dict(k=(BASE + 2, 256, 128)), -5), (dict(v=(BASE, 252, 128)), -5),
    (dict(q=(BASE, 512, 129)), -5), (dict(k=(0, 256, 128)), -1),
    (dict(q_out=(BASE + 16384, 0, 128)), -1), (dict(q_out=(BASE + 16384, 512, 64)), -1),   # writes would collide
    (dict(q_out=(BASE, 1024, 128)), -1),                    # in place with other strides
    (dict(rot=20), -2), (dict(rot=144), -2), (dict(rot=-16), -2), (dict(rope=None), -1), (dict(rope=BASE + 4), -5),
    (dict(rope_rows=999), -3), (dict(inter=2), -1),
])
def test_bad_append_refused(kv8, kw, code):
    kw = {k: (None if v == "null" else kv8.RowsStruct(*v) if isinstance(v, tuple) else v) for k, v in kw.items()}
    assert _append(kv8, _struct(kv8), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), -1), (dict(heads=3), -1), (dict(rows=-1), -1), (dict(max_new=0), -1), (dict(max_new=1001), -3),
    (dict(max_len=0), -1), (dict(max_len=1001), -3), (dict(q="null"), -1), (dict(out="null"), -1),
    (dict(out=(BASE + 16384, 512, 0)), -1), (dict(out=(BASE, 1024, 128)), -1), (dict(q=(BASE + 8, 512, 128)), -5),
    (dict(ws=None), -4), (dict(bytes=1000), -4), (dict(ws=BASE + 128), -5),
    (dict(row_start=None, rows=2), -1), (dict(row_start=BASE + 1), -5),
])
def test_bad_attn_refused(kv8, kw, code):
    kw = {k: (None if v == "null" else kv8.RowsStruct(*v) if isinstance(v, tuple) else v) for k, v in kw.items()}
    assert _attn(kv8, _struct(kv8), **kw) == code


def test_nothing_to_do_is_ok(kv8):
    st = _struct(kv8)
    assert _append(kv8, st, rows=0) == 0 and _append(kv8, st, max_new=0) == 0 and _attn(kv8, st, rows=0) == 0


def test_python_checks(kv8):
    c = kv8.KV8Cache(2, 2, 100, 4, head_dim=64, block=32, dtype=torch.bfloat16, device="cpu")
    assert c.max_blocks == 3 and c.block_table.shape == (2, 3) and (c.block_table == -1).all()
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kv8.kv8_append(c, x.half(), x.half())
    with pytest.raises(ValueError):
        kv8.kv8_append(c, x, x[:1])
    with pytest.raises(ValueError):
        kv8.kv8_append(c, x.transpose(1, 2).contiguous().transpose(1, 2), x)
    with pytest.raises(ValueError):
        kv8.kv8_append(c, x, x, q=x)
    with pytest.raises(ValueError):
        kv8.kv8_append(c, x, x, row_start=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        kv8.kv8_append(c, x, x, rope=torch.zeros(100, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        kv8.KV8Cache(2, 2, 100, 4, seq_len=torch.zeros(2, dtype=torch.int64), device="cpu")
    with pytest.raises(ValueError):
        kv8.KV8Cache(2, 2, 100, 4, fmt="e5m2", device="cpu")
    with pytest.raises(kv8.KvqError):
        kv8.KV8Cache(2, 2, 100, 4, head_dim=80, device="cpu")
    tab = kv8.rope_table(10, 32, device="cpu")
    assert tab.shape == (10, 32)
    np.testing.assert_allclose(tab[7, 3].item(), math.cos(7 * 10000.0 ** (-6 / 32)), rtol=1e-6)
    np.testing.assert_allclose(tab[7, 19].item(), math.sin(7 * 10000.0 ** (-6 / 32)), rtol=1e-6)
