"""Appends with axes, cross attention and attention behind shared prefixes
without a GPU: the oracle's additions against closed forms, and every refusal of
the C ABI and the binding (made before anything is launched)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import kv8 as ok
from test_kv8_cpu import BASE, _struct, kv8  # noqa: F401  (kv8: the fixture)


# ------------------------------------------------------------------ oracle

def test_axes_rows_are_the_pairs_own_positions():
    rng = np.random.default_rng(0)
    table = rng.standard_normal((50, 16))
    axis_of = [0, 2, 1, 1, 0, 2, 2, 0]
    pos = rng.integers(0, 50, (3, 6))
    rows = ok.axes_rows(table, pos, axis_of)
    for r in range(6):
        for i, a in enumerate(axis_of):
            assert rows[r, i] == table[pos[a, r], i] and rows[r, 8 + i] == table[pos[a, r], 8 + i]
    same = ok.axes_rows(table, np.tile(pos[0], (3, 1)), axis_of)
    np.testing.assert_array_equal(same, table[pos[0]])
    pos[1, 2], pos[0, 3] = 50, -1
    bad = np.isnan(ok.axes_rows(table, pos, axis_of))
    assert bad[2].tolist() == [a == 1 for a in axis_of] * 2 and bad[3].tolist() == [a == 0 for a in axis_of] * 2
    assert bad.sum() == 2 * (2 + 3)


def test_axes_turn_by_relative_places():
    """Scores between rotated queries and keys depend on the differences of their
    positions on each axis alone."""
    rng = np.random.default_rng(1)
    half, axis_of = 16, [0] * 4 + [1] * 6 + [2] * 6
    freq = 1.7 ** -np.arange(half)
    ang = np.arange(200)[:, None] * freq
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    x, y = rng.standard_normal((2, 1, 1, 32))
    p, q = rng.integers(0, 90, (2, 3, 1))
    scores = []
    for shift in ([0, 0, 0], [7, 90, 31], [100, 1, 2]):
        s = np.array(shift)[:, None]
        turned = []
        for v, at in ((x, p + s), (y, q + s)):
            row = ok.axes_rows(table, at, axis_of)[0]
            z = (v[0, 0, :half] + 1j * v[0, 0, half:]) * (row[:half] + 1j * row[half:])
            turned.append(z)
        scores.append((turned[0] * turned[1].conj()).real.sum())
    np.testing.assert_allclose(scores, scores[0], rtol=1e-12)


def test_oracle_append_takes_the_rows_own_angles():
    rng = np.random.default_rng(2)
    k, v, q = (ok.round16(rng.standard_normal((9, n, 64)), "float16") for n in (2, 2, 4))
    ang = rng.uniform(0, 6, (9, 16))
    rows = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32).astype(np.float64)
    a, b = (ok.OracleKV8(2, 2, 64, 32, "int8", "float16") for _ in range(2))
    qa = a.append(k, v, [0, 4, 9], None, True, q, rows)
    np.testing.assert_array_equal(qa, ok.rotate(q, rows, True, "float16"))
    np.testing.assert_array_equal(a.k[1], ok.rotate(k[4:], rows[4:], True, "float16"))
    table = np.zeros((9, 32))
    table[:4], table[:5] = rows[:4], rows[4:]
    b.append(k[4:], v[4:], [0, 0, 5], table, True)
    np.testing.assert_array_equal(a.k[1], b.k[1])


def test_oracle_attention_without_order():
    """All rows see all tokens: the textbook formula, whatever the rows' number;
    the newest token's row is the causal one."""
    rng = np.random.default_rng(3)
    k, v = (ok.round16(rng.standard_normal((70, 2, 64)), "float16") for _ in range(2))
    c = ok.OracleKV8(2, 2, 64, 128, "int8", "float16")
    c.append(k, v, [0, 70, 70])
    q = ok.round16(rng.standard_normal((100, 4, 64)), "float16")
    out, bound = c.attention(q, [0, 90, 100], causal=False)
    for i in (0, 5, 89):
        for j in range(4):
            w = np.exp(k[:, j // 2] @ q[i, j] / 8)
            np.testing.assert_allclose(out[i, j], w @ v[:, j // 2] / w.sum(), rtol=1e-12)
    assert (out[90:] == 0).all() and (bound[:90] > 0).all()
    one, _ = c.attention(q[:1], [0, 1, 1])
    np.testing.assert_allclose(out[0], one[0], rtol=1e-12)


# ----------------------------------------------------------------- refusals

def _ref(x):
    return None if x is None else ctypes.byref(x)


def _axes(kv8, st, **kw):
    R = kv8.RowsStruct
    d = dict(k=R(BASE, 256, 128), v=R(BASE, 256, 128), q=R(BASE, 512, 128), q_out=R(BASE, 512, 128), num_q_heads=4,
             row_start=BASE, rows=10, max_new=10, rope=BASE, rope_rows=5, rot_dim=128, interleaved=0, positions=BASE,
             axis_stride=10, num_axes=3, axis_of_pair=bytes([0] * 20 + [1] * 20 + [2] * 24))
    d.update(kw)
    args = kv8.AxesStruct()
    for k, v in d.items():
        if k == "axis_of_pair":
            v = (ctypes.c_uint8 * 64)(*v)
        setattr(args, k, v if v is not None or k not in "kvqq_out" else R(0, 0, 0))
    return kv8.lib.kv8_append_axes(ctypes.byref(st), ctypes.byref(args), None)


def test_axes_struct_layout(kv8):
    """The packed bytes of a call are the struct's."""
    A, R = kv8.AxesStruct, kv8.RowsStruct
    axes = bytes(range(4)) * 16
    rows = [kv8._pack_rows(8 * i + 1, 8 * i + 2, 8 * i + 3) for i in range(4)]
    raw = kv8._pack_axes(*rows, 101, 102, 103, -104, 1, 2, 3, 4, 5, 6, 7, axes)
    x = A.from_buffer_copy(raw)
    for i, t in enumerate((x.k, x.v, x.q, x.q_out)):
        assert (t.data, t.row_stride, t.head_stride) == (8 * i + 1, 8 * i + 2, 8 * i + 3)
    assert (x.row_start, x.rope, x.positions, x.axis_stride) == (101, 102, 103, -104)
    assert (x.num_q_heads, x.rows, x.max_new, x.rope_rows, x.rot_dim, x.interleaved, x.num_axes) == tuple(range(1, 8))
    assert bytes(x.axis_of_pair) == axes and ctypes.sizeof(R) == 24 and ctypes.sizeof(A) == 224
    assert kv8.lib.kv8_append_axes(ctypes.byref(_struct(kv8)), None, None) == -1


def _cross(kv8, st, **kw):
    R = kv8.RowsStruct
    d = dict(heads=4, q=R(BASE, 512, 128), out=R(BASE, 512, 128), row_start=BASE, rows=10, most=10, ws=BASE,
             bytes=1 << 40, max_len=1000)
    d.update(kw)
    return kv8.lib.kv8_cross_attn(ctypes.byref(st), d["heads"], _ref(d["q"]), _ref(d["out"]), d["row_start"],
                                  d["rows"], d["most"], 0.0, d["ws"], d["bytes"], d["max_len"], None)


def _shared(kv8, st, **kw):
    R = kv8.RowsStruct
    d = dict(heads=4, q=R(BASE, 512, 128), out=R(BASE, 512, 128), row_start=BASE, rows=10, max_new=10, groups=BASE,
             prefix=BASE, n=2, most=10, ws=BASE, bytes=1 << 40, max_len=1000)
    d.update(kw)
    return kv8.lib.kv8_shared_attn(ctypes.byref(st), d["heads"], _ref(d["q"]), _ref(d["out"]), d["row_start"],
                                   d["rows"], d["max_new"], d["groups"], d["prefix"], d["n"], d["most"], 0.0, d["ws"],
                                   d["bytes"], d["max_len"], None)


def _args(kv8, kw):
    return {k: (None if v == "null" else kv8.RowsStruct(*v) if isinstance(v, tuple) else v) for k, v in kw.items()}


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=0), -1), (dict(capacity=0), -1), (dict(head_dim=96), -2), (dict(block=16), -2), (dict(dtype=2), -2),
    (dict(num_seqs=65536), -2), (dict(codes=0), -1), (dict(seq_len=0), -1), (dict(block_table=0), -1),
    (dict(codes=BASE + 8), -5), (dict(k_win=BASE + 2), -5), (dict(status=BASE + 2), -5),
])
def test_bad_cache_refused(kv8, kw, code):
    st = _struct(kv8, **kw)
    assert _axes(kv8, st) == code and _cross(kv8, st) == code and _shared(kv8, st) == code


@pytest.mark.parametrize("kw,code", [
    (dict(num_axes=0), -2), (dict(num_axes=5), -2), (dict(num_axes=2), -1),           # the map names a third axis
    (dict(axis_of_pair=bytes([0] * 63 + [4])), -1), (dict(positions=None), -1), (dict(positions=BASE + 2), -5),
    (dict(rot_dim=0), -1), (dict(rot_dim=-16), -1), (dict(rot_dim=24), -2), (dict(rot_dim=144), -2),
    (dict(rope=None), -1), (dict(rope=BASE + 4), -5), (dict(rope_rows=0), -1), (dict(interleaved=2), -1),
    (dict(rows=-1), -1), (dict(max_new=1001), -3), (dict(row_start=BASE + 2), -5), (dict(row_start=None, rows=2), -1),
    (dict(k="null"), -1), (dict(q="null"), -1), (dict(q_out="null"), -1), (dict(num_q_heads=0), -1),
    (dict(v=(BASE, 252, 128)), -5), (dict(q_out=(BASE, 1024, 128)), -1),
])
def test_bad_append_axes_refused(kv8, kw, code):
    assert _axes(kv8, _struct(kv8), **_args(kv8, kw)) == code


def test_append_axes_of_a_smaller_head(kv8):
    """rot_dim above the head dimension is refused, also where the map has room."""
    assert _axes(kv8, _struct(kv8, head_dim=64), k=kv8.RowsStruct(BASE, 128, 64)) == -2


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), -1), (dict(heads=3), -1), (dict(rows=-1), -1), (dict(most=0), -1), (dict(most=-1), -1),
    (dict(most=1 << 30), -2), (dict(max_len=0), -1), (dict(max_len=1001), -3), (dict(q="null"), -1),
    (dict(out="null"), -1), (dict(out=(BASE + 16384, 512, 0)), -1), (dict(out=(BASE, 1024, 128)), -1),
    (dict(q=(BASE + 8, 512, 128)), -5), (dict(ws=None), -4), (dict(bytes=1000), -4), (dict(ws=BASE + 128), -5),
    (dict(row_start=None, rows=2), -1), (dict(row_start=BASE + 1), -5),
])
def test_bad_cross_refused(kv8, kw, code):
    assert _cross(kv8, _struct(kv8), **_args(kv8, kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), -1), (dict(heads=3), -1), (dict(rows=-1), -1), (dict(max_new=0), -1), (dict(max_new=1001), -3),
    (dict(n=0), -1), (dict(n=4), -1), (dict(n=-1), -1), (dict(most=0), -1), (dict(most=1 << 30), -2),
    (dict(groups=None), -1), (dict(prefix=None), -1), (dict(groups=BASE + 2), -5), (dict(prefix=BASE + 1), -5),
    (dict(max_len=0), -1), (dict(max_len=1001), -3), (dict(q="null"), -1), (dict(out="null"), -1),
    (dict(out=(BASE + 16384, 512, 0)), -1), (dict(out=(BASE, 1024, 128)), -1), (dict(q=(BASE + 8, 512, 128)), -5),
    (dict(ws=None), -4), (dict(bytes=1000), -4), (dict(ws=BASE + 128), -5),
    (dict(row_start=None, rows=2), -1), (dict(row_start=BASE + 1), -5),
])
def test_bad_shared_refused(kv8, kw, code):
    assert _shared(kv8, _struct(kv8), **_args(kv8, kw)) == code


def test_nothing_to_do_is_ok(kv8):
    st = _struct(kv8)
    assert _axes(kv8, st, rows=0) == 0 and _axes(kv8, st, max_new=0) == 0
    assert _axes(kv8, st, rows=0, q=None, q_out=None, positions=None) == 0
    assert _axes(kv8, st, rows=0, num_q_heads=0, q=None, q_out=None) == 0
    assert _cross(kv8, st, rows=0) == 0 and _shared(kv8, st, rows=0) == 0


def test_workspace_sizes(kv8):
    """A bound above the capacity is no matter to cross attention; sizes that
    serve more serve less."""
    st = _struct(kv8)
    p, L = ctypes.byref(st), kv8.lib
    assert L.kv8_cross_attn_workspace_bytes(p, 8, 1) >= L.kv8_attn_workspace_bytes(p, 8, 1)
    assert L.kv8_cross_attn_workspace_bytes(p, 8, 5000) > L.kv8_cross_attn_workspace_bytes(p, 8, 1)
    for args in ((7, 1), (8, 0), (8, -1), (8, 1 << 30)):
        assert L.kv8_cross_attn_workspace_bytes(p, *args) == -1
    size = L.kv8_shared_attn_workspace_bytes
    for args in ((7, 10, 1, 5), (8, -1, 1, 5), (8, 10, 0, 5), (8, 10, 1001, 5), (8, 10, 1, 0), (8, 10, 1, 1 << 30)):
        assert size(p, *args) == -1
    last = 0
    for args in ((8, 0, 1, 1), (8, 10, 1, 5), (8, 10, 1, 50), (8, 1000, 1, 50), (8, 1000, 100, 50), (8, 1000, 100, 500)):
        n = size(p, *args)
        assert n % 256 == 0 and n >= last
        last = n
    assert size(p, 8, 10, 1, 5) >= L.kv8_cross_attn_workspace_bytes(p, 8, 1)
    # at least the partial results: 4 D + 8 bytes per row and query head
    assert size(p, 8, 100000, 1, 5) - size(p, 8, 0, 1, 5) >= 100000 * 8 * (4 * 128 + 8)


@pytest.mark.parametrize("D", [64, 128])
def test_workspace_sizes_are_what_they_hold(kv8, D):
    """No more than include/kv8.h says: the sizes of kv8_attn for either part, the
    partial results of the rows, and a few bytes per sequence."""
    for S, Hq, rows, new, most in ((1, 2, 1, 1, 1), (64, 8, 64, 1, 64), (6, 32, 1900, 400, 1900), (3, 2, 900, 900, 30),
                                   (65535, 2, 70000, 2, 500)):
        st = _struct(kv8, num_seqs=S, head_dim=D)
        p, L = ctypes.byref(st), kv8.lib
        own, group = L.kv8_attn_workspace_bytes(p, Hq, new), L.kv8_attn_workspace_bytes(p, Hq, min(most, 1000))
        size = L.kv8_shared_attn_workspace_bytes(p, Hq, rows, new, most)
        rest = size - own - group - (rows * Hq + 32 * 2) * (4 * D + 8)
        assert -32 * 2 * (4 * D + 8) <= rest <= 70 * S + 13000, (S, rest)
        assert 32 * S <= L.kv8_cross_attn_workspace_bytes(p, Hq, new) - own <= 34 * S + 512


def test_python_checks(kv8):
    c = kv8.KV8Cache(2, 2, 100, 4, head_dim=64, block=32, dtype=torch.bfloat16, device="cpu")
    x, ws = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(1 << 20, dtype=torch.uint8)
    rope, pos = kv8.rope_table(10, 64, device="cpu"), torch.zeros(3, 2, dtype=torch.int32)
    axes = kv8.rope_axes([0] * 8 + [1] * 12 + [2] * 12)
    assert axes == bytes([0] * 8 + [1] * 12 + [2] * 12)
    with pytest.raises(ValueError, match="heads"):
        kv8.kv8_append_axes(c, x, x, pos, axes, rope, q=x[:, :0], q_out=x[:, :0])
    for bad in (dict(positions=pos.long()), dict(positions=pos[:, :1]), dict(positions=pos[0]),
                dict(positions=torch.zeros(2, 3, dtype=torch.int32).T), dict(axes=axes[:-1]), dict(axes=list(axes)),
                dict(rope=rope.double()), dict(rope=rope[:, :32]), dict(k=x.half()), dict(q=x),
                dict(row_start=torch.zeros(2, dtype=torch.int32))):
        kw = dict(dict(k=x, v=x, positions=pos, axes=axes, rope=rope), **bad)
        with pytest.raises(ValueError):
            kv8.kv8_append_axes(c, **kw)
    with pytest.raises(ValueError):
        kv8.rope_axes([0, 256])
    with pytest.raises(ValueError, match="CUDA"):
        kv8.kv8_append_axes(c, x, x, pos, axes, rope)
    groups, prefix = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for bad in (dict(group_start=groups[:1]), dict(group_start=groups.long()), dict(prefix_len=prefix.long()),
                dict(prefix_len=prefix[0]), dict(q=x[0]), dict(q=x.half()), dict(out=x[:1]),
                dict(workspace=ws.view(2, -1).T)):
        kw = dict(dict(q=x, out=x, workspace=ws, max_len=10, group_start=groups, prefix_len=prefix, max_group_rows=2),
                  **bad)
        with pytest.raises(ValueError):
            kv8.kv8_shared_attn(c, **kw)
    with pytest.raises(ValueError):
        kv8.kv8_cross_attn(c, x[0], x, ws, 10)
    with pytest.raises(ValueError, match="CUDA"):
        kv8.kv8_cross_attn(c, x, x, ws, 10)
    for f, args in ((kv8.alloc_cross_workspace, (3,)), (kv8.alloc_cross_workspace, (2, 0)),
                    (kv8.alloc_shared_workspace, (2, 10, 101, 5)), (kv8.alloc_shared_workspace, (2, 10, 1, 0))):
        with pytest.raises(kv8.KvqError):
            f(c, *args)
    assert kv8.alloc_shared_workspace(c, 2, 1, 1, 1).dtype == torch.uint8
