"""Appends with positions of several axes, cross attention and attention behind
shared prefixes on the GPU, against the numpy oracle: bit for bit what is
stored, attention within the oracle's bound and half a step of the output's
type.  (Over shared blocks the bound of one pass holds too: weights are rounded
relative to the largest of a part, which is no larger than the row's, and the
join multiplies by powers of two with 2^-22 and adds once, which the bound's
sums of 2^-24 per token and its 2^-15 of a score cover.)"""

import math
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import kv8 as ok
from test_gpu_kv8 import ROOT, TYPES, Run, _dev, _host, kv8  # noqa: F401  (kv8: the fixture)

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------- several axes

class AxesRun(Run):
    """A Run whose tokens have positions on `axes` axes, `top` places each."""

    def __init__(self, kv8, *args, axes=3, axis_of=None, top=300, **kw):
        super().__init__(kv8, *args, **kw)
        self.axes, self.top = axes, top
        self.axis_of = axis_of if axis_of is not None else list(self.rng.integers(0, axes, self.rot // 2))
        self.rope = kv8.rope_table(top, self.rot)
        self.table = _host(self.rope)

    def append(self, new, change=None, implicit=False, positions=None, stride=5):
        H, Hq, D = self.H, self.H * self.g, self.D
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        rows = int(start[-1])
        x = self.numbers((rows, Hq + 2 * H, D))
        x[:, Hq:Hq + H, :: D // 4] *= 4
        if change:
            change(x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:])
        x = ok.round16(x, self.dtype)
        pos = self.rng.integers(0, self.top, (self.axes, rows)) if positions is None else positions
        t = _dev(x, self.dtype)
        buf = torch.full((self.axes, rows + stride), -7, dtype=torch.int32, device="cuda")
        buf[:, :rows] = torch.from_numpy(pos).cuda()
        self.start_host, self.start = start, torch.from_numpy(start).cuda()
        self.q_out = torch.full((rows + 2, Hq, D), 7.0, dtype=t.dtype, device="cuda")
        self.cache.seq_len += _i32(new)
        self.kv8.kv8_append_axes(self.cache, t[:, Hq:Hq + H], t[:, Hq + H:], buf[:, :rows],
                                 self.kv8.rope_axes(self.axis_of), self.rope,
                                 row_start=None if implicit else self.start, max_new=max(1, max(new)), q=t[:, :Hq],
                                 q_out=self.q_out[:rows], interleaved=self.interleaved)
        assert (self.q_out[rows:] == 7.0).all()
        self.q_out = self.q_out[:rows]
        angles = ok.axes_rows(self.table, pos, self.axis_of)
        self.q = self.orc.append(x[:, Hq:Hq + H], x[:, Hq + H:], start, None, self.interleaved, x[:, :Hq], angles)
        return start


@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("D,B", [(128, 32), (128, 64), (128, 128), (64, 32), (64, 64), (64, 128)])
def test_axes_bit_exact(kv8, fmt, dtype, D, B):
    """Prompts, chunks and tokens across block borders, every pair by an axis of
    its own choice; attention over the result."""
    r = AxesRun(kv8, 5, 2, 3, D, B, fmt, dtype, 3 * B + 40, seed=B + D)
    r.append([1, 0, B - 1, 2 * B + 5, B])
    r.check_state()
    r.append([B + 3, 5, 1, 0, 2 * B])
    r.check_state()
    r.append([1] * 5, implicit=True)
    r.check_state()
    r.attend()


@pytest.mark.parametrize("rot,interleaved", [(16, False), (48, True), (64, True), (96, False), (128, True), (128, False)])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("order", ["sections", "turns"])
def test_axes_orders(kv8, rot, interleaved, axes, order):
    """Axes in sections (with borders inside and between four pairs) and in turn."""
    n = rot // 2
    axis_of = [i % axes for i in range(n)] if order == "turns" else [min(i * axes // (n + 3), axes - 1) for i in range(n)]
    r = AxesRun(kv8, 3, 1, 2, 128, 32, "int8", "bfloat16", 200, seed=rot, rot=rot, interleaved=interleaved, axes=axes,
                axis_of=axis_of)
    r.append([40, 64, 3])
    r.check_state()
    r.append([1, 1, 1])
    r.check_state()


@pytest.mark.parametrize("S,H,D,B,fmt,dtype,n", [(3, 11, 64, 32, "int8", "float16", 2300),
                                                 (2, 9, 128, 32, "e4m3", "bfloat16", 14700),
                                                 (3, 9, 128, 64, "int8", "bfloat16", 5900)])
def test_axes_long_prompts(kv8, S, H, D, B, fmt, dtype, n):
    """The forms for many blocks: keys and values apart, eight heads per CTA."""
    r = AxesRun(kv8, S, H, 1, D, B, fmt, dtype, n + 2 * B + 400, seed=n, top=n)
    r.append([B - 3, 0, 7][:S])
    r.append([n - 211 * s for s in range(S)])
    r.check_state()


def test_axes_of_places_are_the_plain_append(kv8):
    """One axis with the tokens' places, and three that agree: kv8_append's bits."""
    for axes in (1, 3):
        a = Run(kv8, 3, 2, 2, 128, 64, "e4m3", "bfloat16", 400, seed=2)
        b = AxesRun(kv8, 3, 2, 2, 128, 64, "e4m3", "bfloat16", 400, seed=2, axes=axes, top=400, axis_of=[i % axes for i in range(64)])
        lens = np.zeros(3, int)
        for new in ([150, 64, 1], [1, 70, 3]):
            b.rng.bit_generator.state = a.rng.bit_generator.state
            a.append(new)
            at = np.concatenate([np.arange(x, x + n) for x, n in zip(lens, new)])
            b.append(new, positions=np.tile(at, (axes, 1)))
            lens += new
            assert torch.equal(a.q_out, b.q_out)
        b.check_state()


def test_axes_that_are_one_line(kv8):
    """Positions expanded from one line (stride 0), as a text's are."""
    r = AxesRun(kv8, 1, 1, 1, 64, 32, "int8", "float16", 100, axes=3, axis_of=[i % 3 for i in range(32)])
    x = _dev(r.numbers((40, 1, 64)), r.dtype)
    line, outs = _i32(r.rng.integers(0, 300, 40)), []
    for pos in (line.expand(3, 40), line.repeat(3, 1)):
        r.cache.seq_len.fill_(40)
        q_out = torch.empty_like(x)
        kv8.kv8_append_axes(r.cache, x, x, pos, kv8.rope_axes(r.axis_of), r.rope, row_start=_i32([0, 40]), max_new=40,
                            q=x, q_out=q_out)
        outs.append((q_out, r.cache.codes[r.cache.block_table[0, 0].long()].clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_axes_positions_beyond_the_capacity(kv8):
    """Positions of a long text in a small cache, rows far apart in the table."""
    r = AxesRun(kv8, 2, 1, 1, 64, 32, "int8", "float16", 100, axes=1, axis_of=[0] * 32, top=70000)
    r.append([60, 33])
    r.check_state()


def test_axes_bad_positions(kv8):
    """A position outside the table: NaN in the channels that turn by it, in the
    row's queries and keys, a status bit, and nothing else.  Rows of no
    sequence may hold any positions."""
    r = AxesRun(kv8, 2, 1, 2, 64, 32, "int8", "float16", 100, axes=2, axis_of=[0] * 8 + [1] * 24, top=50)
    pos = r.rng.integers(0, 50, (2, 40))
    pos[0, 3], pos[1, 5], pos[0, 21], pos[1, 39] = 50, -1, -2 ** 31, 2 ** 31 - 1
    r.append([20, 20], positions=pos)
    assert int(r.cache.status.item()) == 64
    r.cache.status.zero_()
    r.check_state()
    bad = np.isnan(_host(r.q_out))
    assert bad[3, :, :8].all() and bad[3, :, 32:40].all() and bad[3].sum() == 2 * 16 and bad[5].sum() == 2 * 48
    out = np.isnan(_host(r.attend()))
    assert out[3:20].all() and not out[:3].any() and out[21:].all() and not out[20].any()
    # rows behind the sequences', and a sequence that is left out
    r = AxesRun(kv8, 2, 1, 1, 64, 32, "int8", "float16", 100, axes=1, axis_of=[0] * 32, top=10)
    x = _dev(r.numbers((6, 1, 64)), r.dtype)
    q_out = torch.full_like(x, 5.0)
    r.cache.seq_len.copy_(_i32([2, 101]))
    kv8.kv8_append_axes(r.cache, x, x, _i32([[1, 2, 99, 99, -5, 99]]), kv8.rope_axes([0] * 32), r.rope,
                        row_start=_i32([0, 2, 4]), max_new=2, q=x, q_out=q_out)
    assert int(r.cache.status.item()) == 1 and (q_out[2:] == 5.0).all() and not torch.isnan(q_out).any()


def test_axes_in_place_without_queries_and_captured(kv8):
    """q_out is q; no queries; a captured call replayed with other positions."""
    r = AxesRun(kv8, 2, 2, 2, 128, 32, "e4m3", "float16", 100, axes=3, axis_of=[i % 3 for i in range(64)])
    x = [r.numbers((40, n, 128)) for n in (4, 2, 2)]
    q, k, v = (_dev(a, r.dtype) for a in x)
    start = np.array([0, 33, 40], np.int32)
    pos = r.rng.integers(0, 300, (3, 40))
    dpos, dstart, axes = _i32(pos), _i32(start), kv8.rope_axes(r.axis_of)
    r.cache.seq_len += _i32([33, 7])
    kv8.kv8_append_axes(r.cache, k, v, dpos, axes, r.rope, row_start=dstart, max_new=33, q=q, q_out=q)
    r.q = r.orc.append(x[1], x[2], start, None, False, x[0], ok.axes_rows(r.table, pos, r.axis_of))
    r.q_out = q
    r.check_state()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        kv8.kv8_append_axes(r.cache, k[:2], v[:2], dpos[:, :2], axes, r.rope)
    for _ in range(3):
        pos = r.rng.integers(0, 300, (3, 40))
        dpos.copy_(_i32(pos))
        r.cache.seq_len += 1
        g.replay()
        r.orc.append(x[1][:2], x[2][:2], np.arange(3), None, False, None, ok.axes_rows(r.table, pos[:, :2], r.axis_of))
        torch.cuda.synchronize()
        r.check_state()


# ---------------------------------------------------------- cross attention

def cross(r, rows_of, q=None, softmax_scale=0.0, ws=None, implicit=False, check=True, max_len=None):
    """kv8_cross_attn of a Run's cache, rows_of[s] rows for sequence s."""
    start = np.concatenate([[0], np.cumsum(rows_of)]).astype(np.int32)
    rows, Hq = int(start[-1]), r.H * r.g
    q = r.numbers((rows, Hq, r.D)) if q is None else q
    t = _dev(q, r.dtype)
    buf = torch.full((rows + 3, Hq, r.D), 9.0, dtype=t.dtype, device="cuda")
    most = int(max(1, max(rows_of)))
    ws = r.kv8.alloc_cross_workspace(r.cache, Hq, most) if ws is None else ws
    r.kv8.kv8_cross_attn(r.cache, t, buf[:rows], ws, max_len or max(1, max(r.orc.lengths())),
                         row_start=None if implicit else _i32(start), max_rows=most, softmax_scale=softmax_scale)
    torch.cuda.synchronize()
    assert (buf[rows:] == 9.0).all(), "rows behind the last sequence were written"
    if check:
        want, bound = r.orc.attention(q, start, softmax_scale or None, causal=False)
        r.close(_host(buf[:rows]), want, bound)
        assert int(r.cache.status.item()) == 0
    return buf[:rows]


@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("D,B", [(128, 32), (128, 64), (128, 128), (64, 32), (64, 64), (64, 128)])
def test_cross_lengths(kv8, fmt, dtype, D, B):
    """States of every length around units and blocks, none among them; one row
    each, then several, then so many that the tile kernel takes them."""
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 127, 128, 129, 300]
    r = Run(kv8, len(lens), 2, 2, D, B, fmt, dtype, 320, seed=1)
    r.append(lens)
    out = cross(r, [1] * len(lens), implicit=True)
    assert (out[8] == 0).all()
    cross(r, [1] * len(lens), softmax_scale=0.03)
    cross(r, [s % 5 for s in range(len(lens))])
    out = cross(r, [25 if s % 4 == 0 else s % 3 for s in range(len(lens))])  # 50 rows per KV head: the other kernel
    assert (out[25 + 1 + 2 + 0 + 25 + 2 + 0 + 1:][:25] == 0).all()


@pytest.mark.parametrize("H,g", [(1, 1), (3, 1), (2, 5), (2, 8), (1, 9), (1, 16), (1, 17), (1, 49)])
def test_cross_head_layouts(kv8, H, g):
    r = Run(kv8, 3, H, g, 128, 64, "int8", "bfloat16", 400, seed=g)
    r.append([1, 150, 390])
    cross(r, [1, 1, 1])
    cross(r, [3, 4, 0])
    cross(r, [0, 130, 300 // g])


@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("D,g", [(128, 1), (128, 3), (64, 1), (64, 7)])
def test_cross_many_rows(kv8, fmt, dtype, D, g):
    """More rows than tokens, one and two row tiles, many items and cut ones."""
    r = Run(kv8, 4, 2, g, D, 64, fmt, dtype, 2100, seed=4)
    r.append([5, 130, 0, 2050])
    cross(r, [257 // g, 129, 70, 300 // g])


def test_cross_short_and_many(kv8):
    """Hundreds of sequences of a few tokens, which a warp does alone, long ones
    between them that CTAs share, none at all; the same bits every time."""
    S = 300
    r = Run(kv8, S, 2, 2, 64, 32, "e4m3", "float16", 1500, seed=6)
    r.append([1400 if s % 97 == 5 else (7 * s) % 130 for s in range(S)])
    rows = [(1, 2, 0, 3, 9)[s % 5] for s in range(S)]
    q = r.numbers((sum(rows), 4, 64))
    ws = kv8.alloc_cross_workspace(r.cache, 4, 9)
    a = cross(r, rows, q=q, ws=ws)
    for _ in range(3):
        assert torch.equal(a, cross(r, rows, q=q, ws=ws, check=False))
    assert int(ws[:6656].view(torch.int32).abs().sum()) == 0  # the counters


def test_cross_device_errors(kv8):
    """Lengths past the bound give zero rows, bad row ranges leave rows alone,
    a bad block gives NaN; each sets its bit."""
    for g in (1, 60):  # few rows, the other kernel
        r = Run(kv8, 3, 1, g, 64, 32, "int8", "float16", 100)
        r.append([40, 50, 60])
        ws = kv8.alloc_cross_workspace(r.cache, g, 4)
        q = _dev(r.numbers((6, g, 64)), r.dtype)

        def call(start, max_len):
            r.cache.status.zero_()
            out = torch.full_like(q, 3.0)
            kv8.kv8_cross_attn(r.cache, q, out, ws, max_len, row_start=_i32(start), max_rows=2)
            return out, int(r.cache.status.item())

        full, st = call([0, 2, 4, 6], 60)
        assert st == 0
        out, st = call([0, 2, 4, 6], 55)
        assert st == 8 and (out[4:] == 0).all() and torch.equal(out[:4], full[:4])
        out, st = call([0, 2, 4, 7], 60)
        assert st == 2 and (out[4:] == 3.0).all()
        assert g > 1 or torch.equal(out[:4], full[:4])
        out, st = call([0, 3, 4, 6], 60)
        assert st == 2 and (out[:3] == 3.0).all() and torch.equal(out[4:], full[4:])
        out, st = call([0, 2, 1, 3], 60)
        assert st == 2
        r.cache.block_table[1, 0] = -1
        out, st = call([0, 2, 4, 6], 60)
        assert st == 16 and torch.isnan(out[2:4]).all()
        assert torch.equal(out[:2], full[:2]) and torch.equal(out[4:], full[4:])


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("g", [1, 3])
def test_cross_nonfinite(kv8, dtype, g):
    """A NaN or infinite token turns all rows of its sequence and KV head to NaN,
    and no others; a query, its own row."""
    def change(q, k, v):
        v[45, 0, 3] = math.inf
        k[45, 1, 3] = -math.inf

    for rows in ([2, 3], [60, 49]):
        r = Run(kv8, 2, 3, g, 128, 32, "int8", dtype, 200, rot=0)
        r.append([50, 70], change)
        out = np.isnan(_host(cross(r, rows)))
        assert out[: rows[0], : 2 * g].all() and not out[: rows[0], 2 * g:].any() and not out[rows[0]:].any()
        q = r.numbers((sum(rows), 3 * g, 128))
        q[-1, -1, 7] = math.nan
        out = np.isnan(_host(cross(r, rows, q=q)))
        assert out[-1, -1].all() and out[rows[0]:].sum() == 128


def test_cross_in_place_and_strided(kv8):
    """out may be q; rows and heads with strides of their own."""
    r = Run(kv8, 3, 2, 3, 64, 32, "e4m3", "bfloat16", 200, seed=3)
    r.append([100, 31, 190])
    for rows in ([2, 1, 3], [40, 17, 30]):
        n = sum(rows)
        start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        x = r.numbers((n, 9, 64))
        t = _dev(x, r.dtype)
        want, bound = r.orc.attention(x[:, 1:7], start, causal=False)
        ws = kv8.alloc_cross_workspace(r.cache, 6, max(rows))
        wide = torch.full((n, 6, 128), 9.0, dtype=t.dtype, device="cuda")
        kv8.kv8_cross_attn(r.cache, t[:, 1:7], wide[:, :, 64:], ws, 200, row_start=_i32(start), max_rows=max(rows))
        r.close(_host(wide[:, :, 64:]), want, bound)
        assert (wide[:, :, :64] == 9.0).all()
        kv8.kv8_cross_attn(r.cache, t[:, 1:7], t[:, 1:7], ws, 200, row_start=_i32(start), max_rows=max(rows))
        r.close(_host(t[:, 1:7]), want, bound)
        assert torch.equal(t[:, [0, 7, 8]], _dev(x[:, [0, 7, 8]], r.dtype))


def test_cross_of_one_row_each_is_the_last_token_s_attention(kv8):
    """One row per sequence sees what a causal call's newest token sees."""
    r = Run(kv8, 9, 2, 4, 128, 64, "int8", "float16", 700, seed=8)
    r.append([1, 64, 65, 127, 300, 500, 640, 33, 699])
    q = r.numbers((9, 8, 128))
    want, bound = r.orc.attention(q, np.arange(10))
    r.close(_host(cross(r, [1] * 9, q=q)), want, bound)


# ---------------------------------------------------------- shared prefixes

class Groups(Run):
    """A Run whose sequences come in groups that share their first tokens: sizes
    and prefix lengths of the groups, `before` and `behind` sequences of none.
    The others' blocks of those tokens are given up: poison, and no entries."""

    def __init__(self, kv8, sizes, prefixes, H, g, D, B, fmt, dtype, capacity, before=0, behind=0, **kw):
        super().__init__(kv8, before + sum(sizes) + behind, H, g, D, B, fmt, dtype, capacity, **kw)
        self.bounds = before + np.concatenate([[0], np.cumsum(sizes)])
        self.prefixes = prefixes
        lens = np.zeros(self.S, int)
        for x, y, p in zip(self.bounds, self.bounds[1:], prefixes):
            lens[x:y] = p
        start = np.concatenate([[0], np.cumsum(lens)])

        def alike(q, k, v):
            for x, y, p in zip(self.bounds, self.bounds[1:], prefixes):
                for s in range(x + 1, y):
                    for t in (k, v):
                        t[start[s]:start[s] + p] = t[start[x]:start[x] + p]

        if lens.any():
            self.append(list(lens), alike)
        for x, y, p in zip(self.bounds, self.bounds[1:], prefixes):
            if y > x + 1 and p // B:
                lost = self.cache.block_table[x + 1:y, :p // B].flatten().long()
                self.cache.codes.view(torch.uint8)[lost] = 99
                self.cache.scales[lost] = math.nan
                self.cache.block_table[x + 1:y, :p // B] = -1
        self.group_start, self.prefix_len = _i32(self.bounds), _i32(prefixes)

    def most(self, start):
        at = np.asarray(start)[self.bounds]
        return int(max(1, np.diff(at).max()))

    def shared(self, ws=None, check=True, q=None, out=None, softmax_scale=0.0, max_len=None, implicit=False):
        start = self.start_host
        q = self.q if q is None else q
        t = _dev(q, self.dtype)
        rows, Hq = t.shape[0], t.shape[1]
        buf = torch.full((rows + 3, Hq, self.D), 9.0, dtype=t.dtype, device="cuda")
        new, most = int(max(1, np.diff(start).max())), self.most(start)
        if ws is None:
            ws = self.kv8.alloc_shared_workspace(self.cache, Hq, rows, new, most)
        self.kv8.kv8_shared_attn(self.cache, t, buf[:rows], ws, max_len or max(1, max(self.orc.lengths())),
                                 self.group_start, self.prefix_len, most,
                                 row_start=None if implicit else _i32(start), max_new=new,
                                 softmax_scale=softmax_scale)
        torch.cuda.synchronize()
        assert (buf[rows:] == 9.0).all(), "rows behind the last sequence were written"
        if check:
            assert int(self.cache.status.item()) == 0
            want, bound = self.orc.attention(q, start, softmax_scale or None)
            self.close(_host(buf[:rows]), want, bound)
        return buf[:rows]


@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("D,B,g", [(128, 32, 2), (128, 64, 4), (128, 128, 1), (64, 32, 5), (64, 64, 1), (64, 128, 9)])
def test_shared_tokens_and_drafts(kv8, fmt, dtype, D, B, g):
    """Single tokens, then a few at a time: groups of one and of several, with
    prefixes of no block, some, and a part of one more; sequences of no group."""
    r = Groups(kv8, [3, 1, 5, 2], [2 * B + 5, B, 4 * B, B - 1], 2, g, D, B, fmt, dtype, 6 * B + 40, before=1, behind=2,
               seed=B + g)
    r.append([5] + [1, B, 40] + [3] + [1, 2, B + 1, 17, 30] + [0, 2] + [70, 1])
    r.append([1] * r.S, implicit=True)
    r.shared(implicit=True)
    r.shared(softmax_scale=0.03)
    r.append([0, 3, 1, 5, 2, 4, 0, 5, 1, 1, 3, 2, 1, 2])
    r.shared()


@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("D,B,g", [(128, 32, 4), (128, 64, 1), (128, 128, 2), (64, 32, 1), (64, 64, 5), (64, 128, 3)])
def test_shared_chunks(kv8, fmt, dtype, D, B, g):
    """Chunks behind the prefix: the tile kernel on either side, or one of them."""
    r = Groups(kv8, [2, 1, 4], [3 * B, 130, 5 * B + 1], 2, g, D, B, fmt, dtype, 1100, behind=1, seed=8)
    r.append([B - 1, 1, 40, 0, 7, 90, 3, 20])
    r.append([70, 1, 129, 257, 1, 3, 66, 100])
    r.shared()
    r.append([1, 1, 0, 13, 1, 12, 14, 1])
    r.shared()


@pytest.mark.parametrize("D,g,S,prefix", [(128, 8, 36, 2500), (64, 4, 64, 1500), (128, 4, 13, 5000), (64, 16, 2, 6000)])
def test_shared_long_prefix(kv8, D, g, S, prefix):
    """One long prefix, whose keys many CTAs share: all of their parts are joined,
    the same bits every time; the workspace's counters are left zero."""
    r = Groups(kv8, [S], [prefix], 1, g, D, 64, "int8", "bfloat16", prefix + 300, seed=D)
    r.append([(5 * s) % 130 for s in range(S)])
    r.append([1] * S)
    ws = kv8.alloc_shared_workspace(r.cache, g, S, 1, S)
    a = r.shared(ws=ws)
    for _ in range(3):
        assert torch.equal(a, r.shared(ws=ws, check=False))
    assert int(ws[:6656].view(torch.int32).abs().sum()) == 0


def test_shared_many_groups(kv8):
    """More groups and sequences than a warp, or a CTA, looks up at once; empty
    groups; lengths of all kinds."""
    sizes = [(1, 2, 0, 5, 3)[i % 5] for i in range(120)]
    prefixes = [(0, 40, 64, 200, 31)[i % 5] for i in range(120)]
    r = Groups(kv8, sizes, prefixes, 1, 2, 64, 32, "int8", "float16", 420, seed=5, behind=7)
    r.append([(37 * s) % 150 for s in range(r.S)])
    r.append([(1, 0, 3, 1)[s % 4] for s in range(r.S)])
    r.shared()
    sizes = [1] * 500 + [40]
    r = Groups(kv8, sizes, [32] * 500 + [96], 1, 49, 64, 32, "e4m3", "float16", 200, seed=6)
    r.append([s % 40 for s in range(r.S)])
    r.append([1] * r.S)
    r.shared()


def test_shared_equals_the_plain_attention(kv8):
    """With tables that name the same blocks kv8_attn gives the same, within the
    roundings of both."""
    r = Groups(kv8, [4, 3], [256, 100], 2, 4, 128, 64, "int8", "float16", 500, seed=3)
    r.append([1, 30, 100, 64, 5, 6, 7])
    r.append([2, 1, 3, 1, 1, 4, 1])
    a = _host(r.shared())
    for x, y, p in zip(r.bounds, r.bounds[1:], r.prefixes):
        r.cache.block_table[x + 1:y, :p // 64] = r.cache.block_table[x, :p // 64]
    b = _host(r.attend())
    assert np.abs(a - b).max() <= 2.0 ** -9


@pytest.mark.parametrize("g", [2, 30])
def test_shared_device_errors(kv8, g):
    """What only the device sees.  Rows of what is invalid are left alone (zeros
    where a length is above the bound), a status bit is set, others go on."""
    B = 32
    r = Groups(kv8, [3, 2], [2 * B, 3 * B + 1], 1, g, 64, B, "int8", "float16", 300, behind=1, seed=4)
    r.append([5, 0, 40, 3, 33, 50])
    r.append([1, 2, 1, 1, 1, 2])
    start, lens = r.start_host, list(r.orc.lengths())
    q = _dev(r.q, r.dtype)
    ws = kv8.alloc_shared_workspace(r.cache, g, 8, 2, 4)

    def call(group_start=None, prefix=None, rows=4, max_len=300, seq_len=None, row_start=None):
        r.cache.status.zero_()
        r.cache.seq_len.copy_(_i32(lens if seq_len is None else seq_len))
        out = torch.full_like(q, 3.0)
        kv8.kv8_shared_attn(r.cache, q, out, ws, max_len, r.group_start if group_start is None else _i32(group_start),
                            r.prefix_len if prefix is None else _i32(prefix), rows,
                            row_start=_i32(start if row_start is None else row_start), max_new=2)
        torch.cuda.synchronize()
        return out, int(r.cache.status.item())

    full, st = call()
    assert st == 0 and not (full == 3.0).any()
    first, second, last = slice(0, 4), slice(4, 6), slice(6, 8)  # rows of the groups and of the other sequence
    for kw in (dict(prefix=[-1, 3 * B]), dict(prefix=[301, 3 * B]), dict(prefix=[70 + B, 3 * B]), dict(rows=3)):
        out, st = call(**kw)
        assert st == 2 and (out[first] == 3.0).all(), kw
        assert torch.equal(out[second], full[second]) and torch.equal(out[last], full[last]), kw
    # a later sequence that ends within the shared blocks; one above the bound
    short = list(lens)
    short[1] = 2 * B + 1
    out, st = call(seq_len=short)
    assert st == 2 and (out[1:3] == 3.0).all() and torch.equal(out[0], full[0]) and torch.equal(out[3:], full[3:])
    out, st = call(max_len=lens[2] - 1)
    over = [s for s in range(6) if lens[s] > lens[2] - 1]
    assert st == 8 and 2 in over
    for s in range(6):
        rows = slice(start[s], start[s + 1])
        assert (out[rows] == 0).all() if s in over else torch.equal(out[rows], full[rows])
    # bounds that fall, or lie outside: a status bit, nothing out of range
    for kw in (dict(group_start=[0, 4, 3]), dict(group_start=[-1, 3, 5]), dict(group_start=[0, 3, 7]),
               dict(row_start=[0, 2, 1, 4, 5, 6, 8]), dict(row_start=[0, 1, 3, 4, 5, 6, 9]),
               dict(group_start=[5, 0, -3]), dict(group_start=[2 ** 31 - 1, -2 ** 31, 0])):
        assert call(**kw)[1] & 2, kw
    out, st = call()
    assert st == 0 and torch.equal(out, full)
    # an empty group, whatever its prefix
    q_of, prefix = r.prefix_len, _i32([2 * B, 12345, -3, 3 * B + 1])
    r.prefix_len = prefix
    out, st = call(group_start=[0, 3, 3, 3, 5])
    r.prefix_len = q_of
    assert st == 0 and torch.equal(out, full)
    # the first sequence's entry of a shared block
    r.cache.block_table[0, 1] = r.cache.num_blocks
    out, st = call()
    assert st == 16 and torch.isnan(out[first]).all() and torch.equal(out[4:], full[4:])


@pytest.mark.parametrize("new", [1, 30])
@pytest.mark.parametrize("g", [2, 16])
def test_shared_nonfinite(kv8, new, g):
    """A NaN in a shared block turns its group's rows to NaN, one in a sequence's
    own tokens that sequence's; a query its own row and head."""
    r = Groups(kv8, [3, 2], [70, 64], 1, g, 128, 32, "int8", "bfloat16", 200, rot=0, seed=2)

    def change(q, k, v):
        v[12, 0, 5] = math.nan  # sequence 1's

    r.append([10] * 5, change)
    r.append([new] * 5)
    q = r.q.copy()
    q[-1, 1, 3] = math.inf
    out = np.isnan(_host(r.shared(q=q)))
    assert out[new:2 * new].all() and not out[:new].any() and not out[2 * new:-1].any()
    assert out[-1, 1].all() and out[-1].sum() == 128
    r.cache.scales[r.cache.block_table[3, 1].long(), 0, 0] = math.inf
    out = np.isnan(_host(r.shared(check=False)))
    assert out[3 * new:].all() and not out[:new].any() and not out[2 * new:3 * new].any()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("g", [2, 20])
def test_shared_zeros_and_spread_scales(kv8, dtype, g):
    """Blocks of zeros and values of 2^-40 to 2^10 on either side of the prefix's
    end, scores in the hundreds: both parts' sums keep their shares."""
    def spread(which):
        def change(q, k, v):
            q *= 6
            k[:, :, 3] *= 8
            n = len(v)
            if which == "zeros in front":
                v[: n // 2] = 0
            elif which == "zeros behind":
                v[n // 2:] = 0
            elif which == "small in front":
                v[: n // 2] *= 2.0 ** -12
            else:
                v[n // 2:] *= 2.0 ** (-40 if dtype == "bfloat16" else -8)
                v[0] *= 2.0 ** 10
        return change

    for fmt in ("int8", "e4m3"):
        for which in ("zeros in front", "zeros behind", "small in front", "small behind"):
            r = Groups(kv8, [3], [0], 1, g, 128, 32, fmt, dtype, 400, rot=0, seed=3)
            # the prefix by hand, so that its values are changed too
            x = r.numbers((128, 1, 128))
            kk, vv = x.copy(), r.numbers((128, 1, 128))
            spread(which)(np.zeros((128, g, 128)), kk, vv)

            def alike(q, k, v):
                for s in range(3):
                    k[128 * s:128 * s + 128], v[128 * s:128 * s + 128] = kk, vv

            r.append([128] * 3, alike)
            r.cache.block_table[1:, :4] = -1
            r.prefix_len.fill_(128)
            r.append([40, 3, 70], spread(which))
            r.append([1, 2, 1], lambda q, k, v: q.__imul__(6))
            r.shared()


def test_shared_captured_and_replayed(kv8):
    """A captured call is replayed for other lengths, rows and groups within its
    bounds, and on another stream than the tensors' own."""
    r = Groups(kv8, [3, 2], [64, 96], 1, 8, 64, 32, "int8", "float16", 400, seed=7, behind=1)
    r.append([5, 40, 2, 33, 1, 9])
    rows, Hq = 16, 8
    q = torch.zeros((rows, Hq, 64), dtype=torch.float16, device="cuda")
    out, start = torch.zeros_like(q), _i32([0] * 7)
    ws = kv8.alloc_shared_workspace(r.cache, Hq, rows, 4, rows)
    g, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=stream):
        kv8.kv8_shared_attn(r.cache, q, out, ws, 400, r.group_start, r.prefix_len, rows, row_start=start, max_new=4)
    for new, prefix in (([1] * 6, [64, 96]), ([4, 3, 0, 2, 4, 3], [33, 0]), ([0, 0, 1, 0, 0, 0], [64, 64]),
                        ([2, 2, 2, 4, 4, 2], [0, 96])):
        r.append(new)
        n = sum(new)
        start.copy_(_i32(r.start_host))
        r.prefix_len.copy_(_i32(prefix))
        q[:n] = _dev(r.q, r.dtype)
        out.fill_(9.0)
        for x, y, p in zip(r.bounds, r.bounds[1:], r.prefixes):  # what a smaller prefix leaves to each sequence
            r.cache.block_table[x + 1:y, :p // 32] = r.cache.block_table[x, :p // 32]
        for how in ("replayed", "another stream"):
            out.fill_(9.0)
            torch.cuda.synchronize()
            if how == "replayed":
                g.replay()
            else:
                kv8.kv8_shared_attn(r.cache, q, out, ws, 400, r.group_start, r.prefix_len, rows, row_start=start,
                                    max_new=4, stream=torch.cuda.Stream())
            torch.cuda.synchronize()
            assert int(r.cache.status.item()) == 0 and (out[n:] == 9.0).all()
            want, bound = r.orc.attention(r.q, r.start_host)
            r.close(_host(out[:n]), want, bound)


def test_shared_in_place_and_strided(kv8):
    """out may be q; heads in front of rows, and slices of a projection's output."""
    for new in ([1, 1, 1, 1, 1], [30, 2, 1, 20, 1]):
        r = Groups(kv8, [3, 2], [64, 97], 2, 4, 128, 32, "e4m3", "bfloat16", 300, seed=9)
        r.append([5, 40, 2, 33, 1])
        r.append(new)
        n = sum(new)
        want, bound = r.orc.attention(r.q, r.start_host)
        ws = kv8.alloc_shared_workspace(r.cache, 8, n, max(new), n)
        t = torch.full((n, 11, 128), 4.0, dtype=torch.bfloat16, device="cuda")
        t[:, 2:10] = _dev(r.q, r.dtype)
        heads = torch.full((8, n, 128), 4.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        args = (ws, 300, r.group_start, r.prefix_len, n)
        kv8.kv8_shared_attn(r.cache, t[:, 2:10], heads, *args, row_start=r.start, max_new=max(new))
        r.close(_host(heads), want, bound)
        kv8.kv8_shared_attn(r.cache, t[:, 2:10], t[:, 2:10], *args, row_start=r.start, max_new=max(new))
        r.close(_host(t[:, 2:10]), want, bound)
        assert (t[:, [0, 1, 10]] == 4.0).all()


def test_one_workspace_for_all(kv8):
    """kv8_attn, kv8_cross_attn and kv8_shared_attn in turn on one workspace, over
    keys that CTAs' borders cut: the same as with workspaces of their own."""
    calls = []
    for D, S, g, new in ((128, 30, 2, 1), (64, 5, 8, 1), (128, 3, 4, 40), (64, 9, 16, 2)):
        r = Groups(kv8, [S], [2000], 2, g, D, 32, "int8", "float16", 2400, seed=D + S)
        r.append([(11 * s) % 90 for s in range(S)])
        r.append([new] * S)
        r.cache.block_table[1:, :2000 // 32] = r.cache.block_table[0, :2000 // 32]
        q, rows = _dev(r.q, r.dtype), new * S
        start, Hq = _i32(r.start_host), 2 * g

        def run(which, out, ws, r=r, q=q, start=start, new=new, rows=rows):
            if which == 0:
                kv8.kv8_attn(r.cache, q, out, ws, 2400, row_start=start, max_new=new)
            elif which == 1:
                kv8.kv8_cross_attn(r.cache, q, out, ws, 2400, row_start=start, max_rows=new)
            else:
                kv8.kv8_shared_attn(r.cache, q, out, ws, 2400, r.group_start, r.prefix_len, rows, row_start=start,
                                    max_new=new)

        for which in range(3):
            ws = (kv8.alloc_workspace(r.cache, Hq, new), kv8.alloc_cross_workspace(r.cache, Hq, new),
                  kv8.alloc_shared_workspace(r.cache, Hq, rows, new, rows))[which]
            want = torch.full_like(q, 5.0)
            run(which, want, ws)
            calls.append((run, which, want, r, ws.numel()))
    big = torch.zeros(max(c[4] for c in calls), dtype=torch.uint8, device="cuda")
    order = [int(i) for i in np.random.default_rng(0).permutation(len(calls) * 3) % len(calls)]
    for i in order:
        run, which, want, r, _ = calls[i]
        out = torch.full_like(want, 5.0)
        run(which, out, big)
        assert torch.equal(out, want) and int(r.cache.status.item()) == 0, (i, which)
    assert int(big[:6656].view(torch.int32).abs().sum()) == 0


def test_two_streams_with_workspaces_of_their_own(kv8):
    """Calls on two streams at once over one cache, which both only read."""
    r = Groups(kv8, [20], [4000], 2, 8, 128, 64, "int8", "bfloat16", 4300, seed=1)
    r.append([(7 * s) % 100 for s in range(20)])
    r.append([1] * 20)
    q = _dev(r.q, r.dtype)
    want = r.shared(check=False)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    space = [kv8.alloc_shared_workspace(r.cache, 16, 20, 1, 20) for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(8)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(8):
        for j in range(2):
            kv8.kv8_shared_attn(r.cache, q, outs[j][i], space[j], 4300, r.group_start, r.prefix_len, 20,
                                row_start=r.start, stream=streams[j])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for line in outs for o in line)


@pytest.mark.parametrize("new", [1, 30])
def test_pool_past_four_gib(kv8, new):
    """Blocks behind 4 GiB of the pool, for both kernels of either attention, and
    stored there by an append with axes."""
    r = Groups(kv8, [3], [300], 4, 2, 128, 128, "int8", "bfloat16", 600, seed=4, spare=34000)
    assert r.cache.codes.numel() > 2 ** 32 and int(r.cache.block_table.max()) * r.cache.codes[0].numel() > 2 ** 32
    r.append([100, 150, 3])
    r.append([new] * 3)
    r.shared()
    r.cache.block_table[1:, :2] = r.cache.block_table[0, :2]
    cross(r, [new, 2, 1])
    a = AxesRun(kv8, 2, 4, 1, 128, 128, "int8", "bfloat16", 600, seed=5, spare=34000)
    a.append([260, 130])
    tab = a.cache.block_table.cpu().numpy()
    for s, L in enumerate(a.orc.lengths()):
        for b in range(L // 128):
            for h in range(4):
                for j in (0, 1):
                    want, scale = a.orc.block(s, b, h, j == 1)
                    np.testing.assert_array_equal(_host(a.cache.codes[int(tab[s, b]), h, j]), want)
                    assert float(a.cache.scales[int(tab[s, b]), h, j]) == np.float32(scale)


def test_first_calls_of_a_process_are_captured(kv8):
    """Nothing has to run before a capture, for any of the kernels."""
    code = """
import torch
from bit_kv_cache_02_gb300 import kv8
c = kv8.KV8Cache(2, 2, 600, 18, head_dim=128, block=64, fmt="e4m3", dtype=torch.bfloat16)
c.block_table.copy_(torch.arange(18).view(2, 9))
x = torch.randn(400, 8, 128, device="cuda").bfloat16()
q = torch.zeros(400, 4, 128, device="cuda", dtype=torch.bfloat16)
outs = [torch.zeros_like(q) for _ in range(4)]
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
start, late, groups, prefix = i32([0, 300, 400]), i32([0, 100, 101]), i32([0, 2]), i32([64])
pos, rope, axes = torch.arange(400, device="cuda").int().expand(2, 400), kv8.rope_table(600, 128), kv8.rope_axes([0, 1] * 32)
ws, wc = kv8.alloc_shared_workspace(c, 4, 101, 100, 101), kv8.alloc_cross_workspace(c, 4, 100)
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    c.seq_len += start[1:] - start[:-1]
    kv8.kv8_append_axes(c, x[:, 4:6], x[:, 6:], pos, axes, rope, row_start=start, max_new=300, q=x[:, :4], q_out=q)
    kv8.kv8_shared_attn(c, q[:101], outs[0][:101], ws, 600, groups, prefix, 101, row_start=late, max_new=100)
    kv8.kv8_cross_attn(c, q[:101], outs[1][:101], wc, 600, row_start=late, max_rows=100)
g.replay()
kv8.kv8_shared_attn(c, q[:101], outs[2][:101], ws, 600, groups, prefix, 101, row_start=late, max_new=100)
kv8.kv8_cross_attn(c, q[:101], outs[3][:101], wc, 600, row_start=late, max_rows=100)
torch.cuda.synchronize()
assert c.seq_len.tolist() == [300, 100] and int(c.status.item()) == 0
assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
assert all(bool((o[:100] != 0).any(-1).all()) for o in outs[1::2])
print("captured first")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]


def test_wait_that_runs_out(kv8):
    """A wait of the tile kernel that nothing completes ends the call with a
    status, with shared prefixes and in cross attention; the next call on a
    zeroed workspace is right again."""
    from bit_kv_cache_02_gb300 import kvq
    r = Groups(kv8, [4], [640], 1, 16, 128, 64, "int8", "float16", 900, seed=1)
    r.append([30, 1, 2, 3])
    r.append([1] * 4)
    ws = kv8.alloc_shared_workspace(r.cache, 16, 4, 1, 4)
    wc = kv8.alloc_cross_workspace(r.cache, 16, 4)
    for one in (lambda: r.shared(ws=ws, check=False), lambda: cross(r, [4, 4, 4, 4], ws=wc, check=False)):
        assert kvq.lib.kvq_set_wait_test(1000000, 1) == 0
        try:
            one()
            assert int(r.cache.status.item()) & 4
        finally:
            assert kvq.lib.kvq_set_wait_test(0, 0) == 0
        r.cache.status.zero_()
        ws.zero_()
        wc.zero_()
    r.shared(ws=ws)
    for x in r.bounds[:1]:
        r.cache.block_table[x + 1:, :10] = r.cache.block_table[x, :10]
    cross(r, [4, 4, 4, 4], ws=wc)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt,dtype", TYPES)
def test_questions_about_an_image(kv8, fmt, dtype):
    """A decoder layer as a program runs it: a prompt with an image, appended once
    with positions of three axes, is shared by several questions, which are
    appended as chunks and answered token by token, self attention behind the
    shared prefix and cross attention to an encoder's states, two beams each."""
    B, H, g, D, S = 32, 2, 4, 64, 3
    r = AxesRun(kv8, S, H, g, D, B, fmt, dtype, 400, seed=12, axes=3, axis_of=[0] * 8 + [1] * 12 + [2] * 12, top=300)
    enc = Run(kv8, S, H, g, D, B, fmt, dtype, 300, seed=13, rot=0)
    enc.append([150, 0, 277])
    wc = kv8.alloc_cross_workspace(enc.cache, H * g, 2)
    # the prompt, into the first sequence's blocks; the others take them over
    image = np.array([[5, 5 + i // 12, 5 + i % 12] for i in range(96)]).T
    text = np.tile(np.arange(5), (3, 1))
    prompt = np.concatenate([text, image, np.tile(np.arange(17, 48), (3, 1))], 1)  # 132 tokens: four blocks and four
    n = prompt.shape[1]
    r.append([n, 0, 0], positions=prompt)
    full = n // B * B
    for s in range(1, S):
        r.cache.block_table[s, :full // B] = r.cache.block_table[0, :full // B]
        r.cache.k_win[s].copy_(r.cache.k_win[0])
        r.cache.v_win[s].copy_(r.cache.v_win[0])
        r.orc.k[s], r.orc.v[s] = r.orc.k[0].copy(), r.orc.v[0].copy()
    r.cache.seq_len.fill_(n)
    at = np.full(S, 48)
    groups, prefix = _i32([0, S]), _i32([n])
    for new in ([30, 7, 1], [1, 1, 1], [1, 1, 1], [2, 0, 3]):
        pos = np.concatenate([np.tile(np.arange(p, p + k), (3, 1)) for p, k in zip(at, new)], 1)
        at += new
        r.append(new, positions=pos)
        t, rows = r.q_out, sum(new)
        out = torch.full_like(t, 9.0)
        ws = kv8.alloc_shared_workspace(r.cache, H * g, rows, max(new), rows)
        kv8.kv8_shared_attn(r.cache, t, out, ws, 400, groups, prefix, rows, row_start=r.start, max_new=max(new))
        r.close(_host(out), *r.orc.attention(r.q, r.start_host))
        assert int(r.cache.status.item()) == 0
        q = _host(out).repeat(2, 0)[: 2 * S]  # two beams for each of the encoder's sequences
        cross(enc, [2] * S, q=np.ascontiguousarray(q), ws=wc)
