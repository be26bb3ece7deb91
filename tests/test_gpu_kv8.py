"""The 8-bit paged cache on the GPU against the numpy oracle: codes, scales,
windows and rotated queries bit for bit; attention within the bound that the
oracle derives from the kernels' roundings, plus half a step of the output's
type.  Steps are run as a serving loop runs them: raise seq_len, append,
attend."""

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import kv8 as ok

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HALF_STEP = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}  # half a step of subnormals


@pytest.fixture(scope="module")
def kv8():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_kv_cache_02_gb300 import build
    build.build()
    from bit_kv_cache_02_gb300 import kv8 as mod
    return mod


def _dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(getattr(torch, dtype)).cuda()


def _host(t):
    return t.double().cpu().numpy()


class Run:
    """A cache, its oracle and the calls of one test."""

    def __init__(self, kv8, S, H, g, D, B, fmt, dtype, capacity, seed=0, rot=None, interleaved=False, amp=1.0,
                 spare=3):
        self.kv8, self.S, self.H, self.g, self.D, self.B, self.dtype = kv8, S, H, g, D, B, dtype
        self.rng = np.random.default_rng(seed)
        maxb = capacity // B
        # `spare` blocks stay unused; when there are many of them, the first
        self.cache = kv8.KV8Cache(S, H, capacity, max(1, S * maxb + spare), head_dim=D, block=B, fmt=fmt,
                                  dtype=getattr(torch, dtype))
        perm = self.rng.permutation(S * maxb + 3)[: S * maxb].reshape(S, maxb) + spare - 3
        self.cache.block_table.copy_(torch.from_numpy(perm.astype(np.int32)))
        # what no token has been written to must not matter
        self.cache.k_win.fill_(math.nan)
        self.cache.v_win.fill_(math.nan)
        self.cache.scales.fill_(math.nan)
        self.orc = ok.OracleKV8(S, H, D, B, fmt, dtype)
        self.rot = D if rot is None else rot
        self.interleaved = interleaved
        self.rope = kv8.rope_table(capacity, self.rot) if self.rot else None
        self.table = None if self.rope is None else _host(self.rope)
        self.amp = amp
        self.ws = {}

    def numbers(self, shape, amp=1.0):
        return ok.round16(self.rng.standard_normal(shape) * amp, self.dtype)

    def append(self, new, change=None, implicit=False):
        """New tokens per sequence: random q, k, v as slices of one tensor
        (strided), `change` edits them first."""
        H, Hq, D = self.H, self.H * self.g, self.D
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        rows = int(start[-1])
        x = self.numbers((rows, Hq + 2 * H, D), self.amp)
        x[:, Hq:Hq + H, :: D // 4] *= 4
        x = ok.round16(x, self.dtype)
        if change:
            change(x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:])
            x = ok.round16(x, self.dtype)
        t = _dev(x, self.dtype)
        self.start_host, self.start = start, torch.from_numpy(start).cuda()
        self.q_out = torch.full((rows + 2, Hq, D), 7.0, dtype=t.dtype, device="cuda")[:rows]
        self.cache.seq_len += torch.tensor(new, dtype=torch.int32, device="cuda")
        self.kv8.kv8_append(self.cache, t[:, Hq:Hq + H], t[:, Hq + H:], row_start=None if implicit else self.start,
                            max_new=max(1, max(new)), q=t[:, :Hq], q_out=self.q_out, rope=self.rope,
                            interleaved=self.interleaved)
        self.q = self.orc.append(x[:, Hq:Hq + H], x[:, Hq + H:], start, self.table, self.interleaved, x[:, :Hq])
        return start

    def check_state(self):
        c, o, B = self.cache, self.orc, self.B
        assert int(c.status.item()) == 0
        np.testing.assert_array_equal(_host(self.q_out), self.q)
        codes, scales = c.codes.float().cpu().numpy(), c.scales.cpu().numpy()
        kw, vw, tab = _host(c.k_win), _host(c.v_win), c.block_table.cpu().numpy()
        for s, L in enumerate(o.lengths()):
            for h in range(self.H):
                for b in range(L // B):
                    for j in (0, 1):
                        want, scale = o.block(s, b, h, j == 1)
                        np.testing.assert_array_equal(codes[tab[s, b], h, j], want)
                        np.testing.assert_array_equal(scales[tab[s, b], h, j], np.float32(scale))
                r = L % B
                np.testing.assert_array_equal(kw[s, h, :r], o.k[s][L - r:, h])
                np.testing.assert_array_equal(vw[s, h, :r], o.v[s][L - r:, h])

    def attend(self, start=None, q=None, implicit=False, softmax_scale=0.0, ws=None, check=True):
        start = self.start_host if start is None else start
        q = self.q if q is None else q
        t = _dev(q, self.dtype)
        buf = torch.full((t.shape[0] + 3, *t.shape[1:]), 9.0, dtype=t.dtype, device="cuda")
        out = buf[: t.shape[0]]
        new = int(max(1, np.diff(start).max()))
        if ws is None:
            ws = self.kv8.alloc_workspace(self.cache, t.shape[1], new)
        lens = self.orc.lengths()
        self.kv8.kv8_attn(self.cache, t, out, ws, max(1, max(lens)), row_start=None if implicit else
                          torch.from_numpy(np.asarray(start, np.int32)).cuda(), max_new=new,
                          softmax_scale=softmax_scale)
        torch.cuda.synchronize()
        assert (buf[t.shape[0]:] == 9.0).all(), "rows behind the last sequence were written"
        if check:
            want, bound = self.orc.attention(q, start, softmax_scale or None)
            self.close(_host(out), want, bound)
        return out

    def close(self, got, want, bound):
        nan = np.isnan(want)
        np.testing.assert_array_equal(np.isnan(got), nan)
        # the bound of 16 bits counts from the value before its rounding
        tol = bound + HALF_STEP[self.dtype] * (np.abs(want) + bound) + TINY[self.dtype]
        err = np.abs(got - want)[~nan]
        over = err - tol[~nan]
        assert (over <= 0).all(), f"{(over > 0).sum()} of {over.size} off, worst {err[over.argmax()]:.3e} " \
                                  f"with {tol[~nan][over.argmax()]:.3e} allowed"


TYPES = [(f, d) for f in ("int8", "e4m3") for d in ("float16", "bfloat16")]


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("D,B", [(128, 32), (128, 64), (128, 128), (64, 32), (64, 64), (64, 128)])
def test_append_bit_exact(kv8, fmt, dtype, D, B):
    """Prompts of uneven length (one empty), then chunks, then single tokens,
    across block borders."""
    r = Run(kv8, 5, 2, 3, D, B, fmt, dtype, 3 * B + 40, seed=B + D)
    r.append([1, 0, B - 1, 2 * B + 5, B])
    r.check_state()
    r.append([B + 3, 5, 1, 0, 2 * B])
    r.check_state()
    for _ in range(3):
        r.append([1] * 5)
        r.check_state()
    assert sum(n // B for n in r.orc.lengths()) >= 6


@pytest.mark.parametrize("S,H,D,B,fmt,dtype,n", [(3, 11, 64, 32, "int8", "float16", 8300), (2, 9, 128, 32, "e4m3", "bfloat16", 14700),
                                                 (3, 9, 128, 32, "int8", "bfloat16", 2900)])
def test_append_long_prompts(kv8, S, H, D, B, fmt, dtype, n):
    """The forms of the append for many blocks: keys and values by CTAs of their
    own and, from 8192 blocks x heads on, eight heads per CTA, the last ones
    fewer; behind stored tokens, once more behind the result."""
    r = Run(kv8, S, H, 1, D, B, fmt, dtype, n + 2 * B + 400, seed=n)
    r.append([B - 3, 0, 7][:S])
    r.append([n - 211 * s for s in range(S)])
    r.check_state()
    r.append([B + 1] * S)
    r.check_state()


@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, False), (48, True), (64, True), (96, False), (128, True)])
def test_append_rotations(kv8, rot, interleaved):
    r = Run(kv8, 3, 1, 2, 128, 32, "int8", "bfloat16", 200, seed=rot, rot=rot, interleaved=interleaved)
    r.append([40, 64, 3])
    r.check_state()
    r.append([1, 1, 1], implicit=True)
    r.check_state()


@pytest.mark.parametrize("fmt,dtype", TYPES)
def test_append_extreme_values(kv8, fmt, dtype):
    """All zeros, the smallest and largest numbers, one spike, ties, signed zeros."""
    big = 65504.0 if dtype == "float16" else 3.3e38
    tiny = 2.0 ** -24 if dtype == "float16" else 2.0 ** -133

    def change(q, k, v):
        k[0:32], v[0:32] = 0.0, -0.0
        k[32:64], v[32:64] = tiny, -tiny
        k[64:96] = ok.round16(k[64:96] * 1e-3, dtype)
        k[70, 0, 5], v[71, 0, 6] = big, -big
        k[96:128] = np.round(k[96:128] * 4) / 4
        v[96:128] = np.arange(-64, 64)[None, None, :] / 2
        v[96, 0, 0], k[96, 0, 0] = 127.0, 448.0

    r = Run(kv8, 1, 1, 1, 128, 32, fmt, dtype, 200, rot=0)
    r.append([130], change)
    r.check_state()


def test_append_leaves_other_memory_alone(kv8):
    """Blocks and window slots that the call does not reach keep their bytes."""
    r = Run(kv8, 3, 2, 1, 64, 32, "int8", "float16", 160)
    r.append([50, 33, 7])
    before = {n: getattr(r.cache, n).clone() for n in ("codes", "scales", "k_win", "v_win")}
    r.append([0, 30, 1])
    r.check_state()
    tab = r.cache.block_table.cpu().numpy()
    touched = np.zeros(r.cache.num_blocks, bool)
    touched[tab[1, 1]] = True
    for n in ("codes", "scales"):
        x, y = (t[torch.from_numpy(~touched)].contiguous().view(torch.uint8) for t in (before[n], getattr(r.cache, n)))
        assert torch.equal(x.cpu(), y.cpu()), n
    for n in ("k_win", "v_win"):
        x, y = before[n].view(torch.int16).cpu(), getattr(r.cache, n).view(torch.int16).cpu()
        assert torch.equal(x[0], y[0]) and torch.equal(x[2, :, 8:], y[2, :, 8:])


def test_append_in_place_and_transposed(kv8):
    """q_out may be q; k and v may come head-major (any strides)."""
    r = Run(kv8, 2, 2, 2, 128, 32, "e4m3", "float16", 100)
    x = [r.numbers((40, n, 128)) for n in (4, 2, 2)]
    q, k, v = (_dev(a, r.dtype) for a in x)
    k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (k, v))
    start = np.array([0, 33, 40], np.int32)
    r.cache.seq_len += torch.tensor([33, 7], dtype=torch.int32, device="cuda")
    kv8.kv8_append(r.cache, k, v, row_start=torch.from_numpy(start).cuda(), max_new=33, q=q, q_out=q, rope=r.rope)
    r.q, r.q_out = r.orc.append(x[1], x[2], start, r.table, False, x[0]), q
    r.check_state()


def test_append_device_errors(kv8):
    """What only the device sees: nothing is stored for the sequence, its
    status bit is set, the other sequences go on."""
    B = 32
    for case, bit in (("capacity", 1), ("range", 2), ("short", 2), ("block", 16)):
        r = Run(kv8, 2, 1, 1, 64, B, "int8", "float16", 96, rot=0)
        x = _dev(r.numbers((80, 1, 64)), r.dtype)
        start, lens = [0, 40, 80], [40, 40]
        if case == "capacity":
            lens[0] = 97
        elif case == "range":
            start[2] = 81
            start[0] = 0
        elif case == "short":
            lens[0] = 39
        else:
            r.cache.block_table[0, 0] = r.cache.num_blocks
        r.cache.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        codes = r.cache.codes.clone()
        q_out = torch.full_like(x, 5.0)
        kv8.kv8_append(r.cache, x, x, row_start=torch.tensor(start, dtype=torch.int32, device="cuda"), max_new=40,
                       q=x, q_out=q_out)
        torch.cuda.synchronize()
        assert int(r.cache.status.item()) == bit, case
        good = 1 if case != "range" else 0
        bad = 1 - good
        tab = r.cache.block_table.cpu().numpy()
        assert (r.cache.k_win[good, 0, :8] == x[40 * good + 32:40 * good + 40, 0]).all()
        assert not torch.equal(r.cache.codes[tab[good, 0]], codes[tab[good, 0]])
        if case != "block":
            assert torch.isnan(r.cache.k_win[bad]).all()
            assert torch.equal(r.cache.codes[tab[bad, 0]], codes[tab[bad, 0]])
            assert (q_out[40 * bad:40 * bad + 40] == 5.0).all()


@pytest.mark.parametrize("D,B,fmt", [(128, 32, "int8"), (64, 64, "e4m3"), (128, 128, "e4m3")])
def test_append_one_row_each_under_a_larger_bound(kv8, D, B, fmt):
    """Without row_start every sequence brings one row, also where max_new is
    the bound of the whole program, above the block: steps across block borders,
    with rows of no sequence behind, then attention by the same arguments."""
    S, g, most = 4, 2, 2 * B + 30
    r = Run(kv8, S, 2, g, D, B, fmt, "float16", 4 * B, seed=B)
    r.append([B - 2, 0, 2 * B - 1, 5])
    start = np.arange(S + 1)
    for _ in range(3):
        x = r.numbers((S + 2, 2 * g + 4, D))
        t = _dev(x, r.dtype)
        q_out = torch.full((S + 2, 2 * g, D), 5.0, dtype=t.dtype, device="cuda")
        out = q_out.clone()
        r.cache.seq_len += 1
        kv8.kv8_append(r.cache, t[:, 2 * g:2 * g + 2], t[:, 2 * g + 2:], max_new=most, q=t[:, :2 * g], q_out=q_out,
                       rope=r.rope)
        r.q = r.orc.append(x[:S, 2 * g:2 * g + 2], x[:S, 2 * g + 2:], start, r.table, False, x[:S, :2 * g])
        r.q_out = q_out[:S]
        r.check_state()
        kv8.kv8_attn(r.cache, q_out, out, kv8.alloc_workspace(r.cache, 2 * g, most), 4 * B, max_new=most)
        r.close(_host(out[:S]), *r.orc.attention(r.q, start))
        assert (q_out[S:] == 5.0).all() and (out[S:] == 5.0).all()


# --------------------------------------------------------------- attention

@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("D,B", [(128, 32), (128, 64), (128, 128), (64, 32), (64, 64), (64, 128)])
def test_token_lengths(kv8, fmt, dtype, D, B):
    """One query per sequence; lengths around every unit and block border."""
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300]
    r = Run(kv8, len(lens), 2, 2, D, B, fmt, dtype, 320, seed=1)
    r.append([n - 1 for n in lens])
    r.append([1] * len(lens), implicit=True)
    r.check_state()
    r.attend()
    r.attend(implicit=True, softmax_scale=0.03)


@pytest.mark.parametrize("H,g", [(1, 1), (3, 1), (2, 5), (2, 8), (1, 9), (1, 16), (1, 17), (1, 40)])
def test_token_head_layouts(kv8, H, g):
    r = Run(kv8, 3, H, g, 128, 64, "int8", "bfloat16", 400, seed=g)
    r.append([1, 150, 390])
    r.append([1, 1, 1])
    r.attend()


@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("D,g,new", [(128, 4, [3, 8, 1, 0, 5]), (64, 1, [16, 9, 2, 1, 0]), (128, 2, [60, 1, 33, 7, 64]),
                                     (64, 7, [40, 1, 1, 3, 0]), (128, 1, [150, 0, 129, 1, 3])])
def test_several_tokens(kv8, fmt, dtype, D, g, new):
    """Drafts, chunks and mixed batches: every row up to its own position."""
    r = Run(kv8, 5, 2, g, D, 32, fmt, dtype, 400, seed=3)
    r.append([0, 70, 1, 200, 31])
    r.append(new)
    r.check_state()
    r.attend()


@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("D,B,g", [(128, 32, 4), (128, 64, 1), (128, 128, 2), (64, 32, 1), (64, 64, 5), (64, 128, 3)])
def test_chunks(kv8, fmt, dtype, D, B, g):
    """Chunks of more rows than the rows kernel takes: one and two row tiles,
    prefixes of none to many units, partly filled last blocks and windows."""
    r = Run(kv8, 6, 2, g, D, B, fmt, dtype, 700, seed=8)
    r.append([0, 1, B, 130, 400, 299])
    r.append([70, 129, 65 + B, 257, 128, 300])
    r.check_state()
    r.attend()


def test_chunk_layouts(kv8):
    """Query groups that do not divide the row tiles, many items for few CTAs
    and few items for many."""
    for H, g, ctx, new in ((1, 17, [40, 0, 300], [60, 5, 100]), (9, 1, [0] * 3, [129, 70, 200]),
                           (1, 1, [5000], [90]), (1, 3, [0, 0, 0, 0], [300, 0, 100, 1])):
        r = Run(kv8, len(ctx), H, g, 128, 64, "int8", "bfloat16", 6000, seed=g)
        r.append(ctx)
        r.append(new)
        ws = kv8.alloc_workspace(r.cache, H * g, max(new))
        a = r.attend(ws=ws)
        assert torch.equal(a, r.attend(ws=ws, check=False)), "a repeated call gave another result"


def test_many_chunks_at_once(kv8):
    """More sequences with rows for the tile kernel than it has threads to look
    them up at once, empty ones among them."""
    S = 700
    r = Run(kv8, S, 1, 49, 64, 32, "int8", "float16", 100, seed=9)
    r.append([(37 * s) % 70 for s in range(S)])
    r.append([(1, 1, 0, 1, 6)[s % 5] for s in range(S)])
    assert r.start_host[-1] * 49 // 256 + S > 768
    r.attend()


@pytest.mark.parametrize("D", [64, 128])
def test_weights_follow_each_other_under_a_still_maximum(kv8, D):
    """All scores alike, so that from the second unit on the maximum does not
    move and weights follow weights with nothing but the wait between them;
    values differ by unit, so that a weight stored too early or too late shows.
    The same bits every time."""
    def change(q, k, v):
        k[:] = 0.5
        v[:] = (np.arange(len(v)) // 128 % 7 - 3.0)[:, None, None] + np.sign(v) / 4

    r = Run(kv8, 1, 2, 2, D, 64, "e4m3", "float16", 6000, rot=0)
    r.append([5000], change)
    r.append([128], change)
    ws = kv8.alloc_workspace(r.cache, 4, 128)
    want = r.attend(ws=ws)
    for _ in range(50):
        assert torch.equal(want, r.attend(ws=ws, check=False))


@pytest.mark.parametrize("fmt,dtype", TYPES)
def test_rows_without_keys_get_zeros(kv8, fmt, dtype):
    """More rows than tokens, and sequences without a token; with more query
    heads the same rows take the other kernel."""
    for g in (2, 9):
        _rows_without_keys(kv8, fmt, dtype, g)


def _rows_without_keys(kv8, fmt, dtype, g):
    r = Run(kv8, 3, 1, g, 64, 32, fmt, dtype, 100)
    r.append([5, 0, 40])
    start = np.array([0, 9, 12, 60], np.int32)
    q = r.numbers((60, g, 64))
    out = _host(r.attend(start, q))
    assert (out[0:4] == 0).all() and (out[9:12] == 0).all() and (out[12:20] == 0).all()
    assert (out[4] != 0).any() and (out[20] != 0).any()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("where", ["window", "block"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("g", [1, 3])
def test_nonfinite_tokens(kv8, dtype, where, value, g):
    """NaN in the rows that see a NaN or infinite token (its block, once
    quantized), nothing in the others; a later, hidden one does no harm."""
    B = 32
    at = 45 if where == "window" else 20

    for which in (0, 1):
        def change(q, k, v):
            (k, v)[which][at, 0, 3] = value
            (k, v)[which][at, 0, 64] = value

        r = Run(kv8, 1, 2, g, 128, B, "int8", dtype, 200, rot=0)
        r.append([50], change)
        out = _host(r.attend())
        first = at if where == "window" else 0
        assert np.isnan(out[first:, :g]).all() and not np.isnan(out[:, g:]).any()
        assert not np.isnan(out[:first]).any()


@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_nonfinite_queries(kv8, fmt, dtype, value):
    """A query with a NaN or an infinity gives NaN in its own row and head (zeros
    where it sees no token), also where it makes every score -infinity."""
    def change(q, k, v):
        k[:, :, 3] = 1 + np.abs(k[:, :, 3])  # an infinite channel has one sign for all tokens

    for ctx, new in ((70, 1), (70, 12), (64, 70), (5000, 1), (5000, 100)):
        r = Run(kv8, 1, 2, 3, 128, 64, fmt, dtype, 5200, rot=0)
        r.append([ctx], change)
        r.append([new], change)
        q = r.q.copy()
        q[new // 2, 1, 3] = q[0, 4, 3] = value
        out = _host(r.attend(q=q))  # the oracle's NaN are those two heads
        assert np.isnan(out[new // 2, 1]).all() and np.isnan(out[0, 4]).all() and np.isnan(out).sum() == 2 * 128
    r = Run(kv8, 1, 1, 3, 64, 32, fmt, dtype, 100)
    r.append([5])
    q = r.numbers((30, 3, 64))
    q[3, 1, 3] = value
    out = _host(r.attend(np.array([0, 30]), q))
    assert (out[3] == 0).all() and not np.isnan(out).any()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_large_scores_and_spread_scales(kv8, dtype):
    """Scores in the hundreds, blocks whose scales differ by 2^20, window
    tokens far larger and far smaller than their neighbours."""
    def change(q, k, v):
        q *= 8
        k[:, :, 3] *= 8
        v[0:32] *= 2.0 ** -10
        v[32:64] *= 2.0 ** 10
        v[96:100] *= 2.0 ** -8
        v[101] *= 2.0 ** 9

    for fmt in ("int8", "e4m3"):
        r = Run(kv8, 1, 1, 4, 128, 32, fmt, dtype, 200, rot=0)
        r.append([110], change)
        r.check_state()
        r.attend()
        r.append([3])  # few rows
        r.attend()


def test_blocks_of_zeros(kv8):
    """Values of zero have no scale to speak of, and their tokens still weigh."""
    def change(q, k, v):
        v[:96] = 0
        k[:32] = 0

    for dtype in ("float16", "bfloat16"):
        r = Run(kv8, 1, 1, 2, 128, 32, "int8", dtype, 200, rot=0)
        r.append([140], change)
        r.attend()
        r.append([1])
        r.attend()


def test_many_sequences_and_splits(kv8):
    """More sequences than a warp scans at once, and one long sequence whose
    keys many CTAs share; a workspace is reused across shapes."""
    r = Run(kv8, 150, 1, 2, 64, 32, "int8", "float16", 260, seed=5)
    lens = [(37 * s) % 250 for s in range(150)]
    r.append(lens)
    ws = kv8.alloc_workspace(r.cache, 2, 4)
    r.append([1] * 150)
    r.attend(ws=ws)
    r.append([(s * 7) % 4 for s in range(150)])
    r.attend(ws=ws)
    r2 = Run(kv8, 1, 1, 1, 64, 32, "e4m3", "bfloat16", 20000, seed=6)
    r2.append([19000])
    r2.append([1])
    a = r2.attend(ws=ws)
    for _ in range(3):
        assert torch.equal(a, r2.attend(ws=ws, check=False)), "a repeated call gave another result"
    assert int(ws[-2560:].view(torch.int32).abs().sum()) == 0


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_workspace_serves_other_shapes(kv8, dtype):
    """One workspace for caches of both head dimensions in turn, single tokens
    and chunks over keys that all CTAs' borders cut: the same as with workspaces
    of their own.  What one call leaves of its partial results is no other
    call's counter."""
    dt = getattr(torch, dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    calls = []
    for D in (128, 64):
        L, H, B = 15000, 8, 64
        c = kv8.KV8Cache(1, H, L, L // B, head_dim=D, block=B, fmt="e4m3", dtype=dt)
        for j in range(2):
            c.codes[:, :, j] = torch.randn(c.codes[:, :, j].shape, generator=gen, device="cuda").to(c.codes.dtype)
        c.scales.fill_(1.0)
        for win in (c.k_win, c.v_win):
            win.copy_(torch.randn(win.shape, generator=gen, device="cuda"))
        c.block_table.copy_(torch.arange(L // B, device="cuda"))
        c.seq_len.fill_(L)
        for new in (1, 5, 130):
            q = torch.randn((new, H, D), generator=gen, device="cuda").to(dt)
            start = torch.tensor([0, new], dtype=torch.int32, device="cuda")
            want = torch.full_like(q, 5.0)
            kv8.kv8_attn(c, q, want, kv8.alloc_workspace(c, H, new), L, row_start=start, max_new=new)
            calls.append((c, q, start, new, want))
    ws = kv8.alloc_workspace(calls[0][0], 8, 130)
    for i in (0, 3, 0, 5, 0, 2, 5, 2, 3, 1, 4, 1, 5, 4, 2):
        c, q, start, new, want = calls[i]
        out = torch.full_like(q, 5.0)
        kv8.kv8_attn(c, q, out, ws, c.capacity, row_start=start, max_new=new)
        assert torch.equal(out, want) and int(c.status.item()) == 0
    assert int(ws[:3328].view(torch.int32).abs().sum()) == 0  # the counters


def test_attn_device_errors(kv8):
    """Lengths past the bound give zero rows, bad row ranges leave rows alone,
    a bad block gives NaN; each sets its bit."""
    r = Run(kv8, 3, 1, 1, 64, 32, "int8", "float16", 100)
    r.append([40, 50, 60])
    ws = kv8.alloc_workspace(r.cache, 1, 4)
    q = _dev(r.numbers((6, 1, 64)), r.dtype)

    def call(start, max_len, max_new=2):
        r.cache.status.zero_()
        out = torch.full_like(q, 3.0)
        kv8.kv8_attn(r.cache, q, out, ws, max_len, row_start=torch.tensor(start, dtype=torch.int32, device="cuda"),
                     max_new=max_new)
        return out, int(r.cache.status.item())

    full, st = call([0, 2, 4, 6], 60)
    assert st == 0
    out, st = call([0, 2, 4, 6], 55)
    assert st == 8 and (out[4:] == 0).all() and torch.equal(out[:4], full[:4])
    out, st = call([0, 2, 4, 7], 60)
    assert st == 2 and (out[4:] == 3.0).all() and torch.equal(out[:4], full[:4])
    out, st = call([0, 2, 1, 3], 60)
    assert st == 2
    out, st = call([0, 3, 4, 6], 60)
    assert st == 2 and (out[:3] == 3.0).all() and torch.equal(out[4:], full[4:])
    r.cache.block_table[1, 0] = -1
    out, st = call([0, 2, 4, 6], 60)
    assert st == 16 and torch.isnan(out[2:4]).all() and torch.equal(out[:2], full[:2]) and torch.equal(out[4:], full[4:])


def test_shared_blocks(kv8):
    """Two sequences whose tables name the same blocks (a shared prefix)."""
    r = Run(kv8, 2, 1, 2, 128, 32, "int8", "float16", 128, rot=0)
    x = r.numbers((64, 1, 128))

    def change(q, k, v):
        k[64:], v[64:] = k[:64], v[:64]

    r.append([64, 64], change)
    r.cache.block_table[1] = r.cache.block_table[0]
    r.append([3, 1])
    r.attend()
    assert x.shape[0] == 64


def test_blocks_behind_a_changed_table(kv8):
    """A sequence whose table is changed to another's blocks sees those, and
    nothing of the blocks that it had, whatever is in them now."""
    for new in (1, 30):  # few rows, the other kernel
        r = Run(kv8, 2, 1, 2, 128, 32, "int8", "float16", 160, rot=0)
        r.append([64, 64])
        own = r.cache.block_table[1, :2].long()
        r.cache.block_table[1, :2] = r.cache.block_table[0, :2]
        r.cache.codes[own] = 99
        r.cache.scales[own] = math.nan
        r.orc.k[1], r.orc.v[1] = r.orc.k[0].copy(), r.orc.v[0].copy()
        r.append([3, new])
        r.attend()


def test_capacity_below_a_block(kv8):
    """A cache whose tokens never fill a block needs no pool."""
    for new in (1, 25):
        r = Run(kv8, 2, 2, 3, 64, 128, "int8", "bfloat16", 90, spare=3)
        assert r.cache.max_blocks == 0
        for name in ("codes", "scales", "block_table"):
            setattr(r.cache.struct, name, None)
        r.append([40, 0])
        r.append([new, 20])
        r.attend()
        assert int(r.cache.status.item()) == 0


@pytest.mark.parametrize("H,g", [(1, 49), (2, 72), (1, 300)])
def test_token_many_query_heads(kv8, H, g):
    """Query groups so large that a single token's rows take the other kernel."""
    r = Run(kv8, 3, H, g, 128, 64, "int8", "float16", 400, seed=g)
    r.append([1, 150, 390])
    r.append([1, 1, 1], implicit=True)
    r.attend(implicit=True)
    r.attend()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_tiny_values(kv8, fmt):
    """bf16 values near 2^-100, in blocks before normal ones and in the window:
    the normalizer, which divides by their scale, stays finite.  A block whose
    scale is below 2^-80 counts as zeros: its values are below 448 * 2^-80, and
    so is what the weighted sum loses."""
    def change(q, k, v):
        v[:640] = 2.0 ** -99 * np.sign(v[:640])
        v[704:708] = 2.0 ** -110

    for lead in (640, 704, 720):
        r = Run(kv8, 1, 1, 2, 128, 32, fmt, "bfloat16", 800, rot=0)
        r.append([lead], change)
        r.append([3])
        want, bound = r.orc.attention(r.q, r.start_host)
        r.close(_host(r.attend(check=False)), want, bound + 448 * 2.0 ** -80)
        r.append([40])  # rows enough for the other kernel
        want, bound = r.orc.attention(r.q, r.start_host)
        r.close(_host(r.attend(check=False)), want, bound + 448 * 2.0 ** -80)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("e", [-60, -40, 0, 70, 90])
@pytest.mark.parametrize("first", [True, False])
def test_zero_blocks_beside_small_and_large_values(kv8, fmt, e, first):
    """bf16 values around 2^e and, before or behind them, blocks whose values are
    zero, in one CTA's part and in parts that are merged: neither the small
    values' bits nor the zeros' share of the weights are lost.  (The bound is
    relative to the values.)"""
    def scaled(q, k, v):
        v *= 2.0 ** e

    def zeroed(q, k, v):
        v[:] = 0

    for long in (0, 4000):
        r = Run(kv8, 1, 1, 1, 128, 32, fmt, "bfloat16", 8448, rot=0)
        r.append([96 + long], zeroed if first else scaled)
        r.append([96 + long], scaled if first else zeroed)
        for steps in ([64], [32], [24, 8]):  # the tile kernel, up to sixteen rows at once, up to eight
            for new in steps:
                r.append([new], scaled)
            r.attend()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("e", [-60, -40, 0, 70, 90])
def test_windows_of_zero_small_and_large_values(kv8, fmt, e):
    """The same where the window holds such tokens, zeros among them, and where
    hidden tokens of the window are far larger."""
    def scaled(q, k, v):
        v *= 2.0 ** e
        v[1::3] = 0

    def last_large(q, k, v):
        scaled(q, k, v)
        v[-1] *= 2.0 ** (95 - max(e, 0) - 6)

    for long in (0, 4000):
        for change in (scaled, last_large):
            r = Run(kv8, 1, 1, 1, 128, 64, fmt, "bfloat16", 8448, rot=0)
            r.append([96 + long], scaled)
            for new in (63, 15, 3):  # the tile kernel, up to sixteen rows at once, up to eight
                r.append([new], change)
                r.attend()
                r.append([64 + 30 - (new + 30) % 64], scaled)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,B,g", [(128, 32, 1), (64, 64, 3), (128, 64, 9), (64, 32, 20)])
def test_values_of_all_sizes_side_by_side(kv8, fmt, D, B, g):
    """bf16 values of 2^-60 to 2^60 by token or by sixteen tokens, zeros among
    them, so that rows see small tokens of blocks whose hidden ones are large:
    within the bound, whose subnormals' part counts every token's unit."""
    for seed, run in ((1, 1), (2, 16)):
        r = Run(kv8, 3, 2, g, D, B, fmt, "bfloat16", 700, seed=seed, rot=0)

        def change(q, k, v):
            e = r.rng.integers(-60, 61, len(v) // run + 1).repeat(run)[:len(v)]
            v *= np.where(r.rng.random(len(v)) < 0.2, 0.0, 2.0 ** e)[:, None, None]

        r.append([2 * B + 5, 0, 300], change)
        for new in ([70, 1, 100], [3, 1, 8], [1, 1, 1]):
            r.append(new, change)
            r.check_state()
            r.attend()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_long_context_precision(kv8, fmt):
    """Over a long context of independent values the sums nearly cancel, and the
    elements' bound says little.  Each weight is off by at most 2^-11 of itself,
    independently, so the error's 2-norm is at most 2^-11 of the output's; the
    output's own rounding adds 2^-11 of each element: together 2^(1/2) 2^-11,
    and 2^-10 leaves a factor of 2^(1/2) for chance and the fp32 sums."""
    r = Run(kv8, 1, 1, 4, 128, 64, fmt, "float16", 20000, seed=2, rot=0)
    r.append([19800])
    for new in (1, 3, 40):  # few rows, more rows, the other kernel
        r.append([new])
        want, _ = r.orc.attention(r.q, r.start_host)
        got = _host(r.attend(check=False))
        err = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert err <= 2.0 ** -10, f"{new} tokens: {err:.2e}"


def test_pool_past_four_gigabytes(kv8):
    """Offsets into the pool need more than 32 bits: 16,500 unused blocks of 256
    KiB come first."""
    r = Run(kv8, 2, 8, 2, 128, 128, "int8", "float16", 600, spare=16500)
    assert r.cache.codes.numel() > 2 ** 32
    r.append([500, 130])
    r.attend()
    r.append([1, 1])
    r.attend()
    r.append([3, 30])
    r.attend()


def test_rows_before_the_first_sequence(kv8):
    """row_start may begin behind row 0; rows of no sequence stay as they are."""
    B, pad = 32, 70
    for new in ([1, 1], [3, 9], [100, 40]):
        r = Run(kv8, 2, 2, 3, 128, B, "e4m3", "float16", 300)
        r.append([45, 0])
        start = np.concatenate([[0], np.cumsum(new)])
        x = r.numbers((start[-1] + 2 * pad, 10, 128))
        t = _dev(x, r.dtype)
        q_out = torch.full((len(x), 6, 128), 5.0, dtype=t.dtype, device="cuda")
        out = q_out.clone()
        rs = torch.from_numpy((start + pad).astype(np.int32)).cuda()
        r.cache.seq_len += torch.tensor(new, dtype=torch.int32, device="cuda")
        kv8.kv8_append(r.cache, t[:, 6:8], t[:, 8:], row_start=rs, max_new=max(new), q=t[:, :6], q_out=q_out, rope=r.rope)
        mid = slice(pad, pad + start[-1])
        r.q = r.orc.append(x[mid, 6:8], x[mid, 8:], start, r.table, False, x[mid, :6])
        r.q_out = q_out[mid]
        r.check_state()
        kv8.kv8_attn(r.cache, q_out, out, kv8.alloc_workspace(r.cache, 6, max(new)), 300, row_start=rs, max_new=max(new))
        r.close(_host(out[mid]), *r.orc.attention(r.q, start))
        for y in (q_out, out):
            assert (y[:pad] == 5.0).all() and (y[pad + start[-1]:] == 5.0).all()


def test_output_in_place(kv8):
    """out may be q: single tokens, parts of a long line, items cut by CTAs."""
    for ctx, new in (([300, 5], [1, 1]), ([5000, 3], [2, 4]), ([5000, 200], [90, 30])):
        r = Run(kv8, 2, 2, 2, 128, 64, "int8", "bfloat16", 6000, rot=0)
        r.append(ctx)
        r.append(new)
        want = r.attend()
        q = r.q_out.clone()
        kv8.kv8_attn(r.cache, q, q, kv8.alloc_workspace(r.cache, 4, max(new)), max(r.orc.lengths()), row_start=r.start,
                     max_new=max(new))
        assert torch.equal(q, want)


def test_falling_row_start(kv8):
    """Row ranges that go back set the status; nothing outside the tensors is
    touched and rows of no sequence stay as they are."""
    r = Run(kv8, 3, 1, 1, 64, 32, "int8", "float16", 200, rot=0)
    x = _dev(r.numbers((200, 1, 64)), r.dtype)
    r.cache.seq_len.fill_(150)
    rs = torch.tensor([0, 150, 90, 150], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 5.0)
    kv8.kv8_append(r.cache, x, x, row_start=rs, max_new=150, q=x, q_out=out)
    assert int(r.cache.status.item()) == 2
    assert (out[150:] == 5.0).all()
    r.cache.status.zero_()
    kv8.kv8_attn(r.cache, x, out, kv8.alloc_workspace(r.cache, 1, 150), 150, row_start=rs, max_new=150)
    assert int(r.cache.status.item()) & 2
    assert (out[150:] == 5.0).all()


def test_wait_that_runs_out(kv8):
    """The tile kernel's waits are bounded.  Here the keys of each CTA's second
    unit wait, with a limit of 20000 SM cycles, for a barrier that nothing
    completes: all roles leave, the products under way drain, tensor memory is
    given back, the status says so and the device stays usable.  On a workspace
    that is zero again the same call is right."""
    from bit_kv_cache_02_gb300 import kvq
    for D, ctx, new in ((128, [5000, 100], [200, 1]), (64, [0, 700], [300, 90])):
        r = Run(kv8, 2, 2, 2, D, 64, "int8", "bfloat16", 5400, rot=0)
        r.append(ctx)
        r.append(new)
        ws = kv8.alloc_workspace(r.cache, 4, max(new))
        try:
            kvq.set_wait_test(20000, True)
            for _ in range(3):
                r.attend(ws=ws, check=False)
                assert int(r.cache.status.item()) == kvq.KVQ_STATUS_TIMEOUT
                r.cache.status.zero_()
        finally:
            kvq.set_wait_test(0, False)
        ws.zero_()
        r.attend(ws=ws)
        assert int(r.cache.status.item()) == 0


# -------------------------------------------------------- streams and graphs

def test_two_streams_at_once(kv8):
    """Two caches with workspaces of their own on two streams: the same results
    as one after the other."""
    runs = []
    for i, (D, new) in enumerate(((128, [300, 80]), (64, [90, 1]))):
        r = Run(kv8, 2, 2, 2, D, 32, "int8", "float16", 1000, seed=i)
        r.append([400, 100])
        r.append(new)
        q, ws = r.q_out.clone(), kv8.alloc_workspace(r.cache, 4, max(new))
        runs.append((r, q, ws, max(new), r.attend(), torch.zeros_like(q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for r, q, ws, new, _, out, stream in runs:
            kv8.kv8_attn(r.cache, q, out, ws, max(r.orc.lengths()), row_start=r.start, max_new=new, stream=stream)
    torch.cuda.synchronize()
    for r, _, _, _, want, out, _ in runs:
        assert torch.equal(out, want) and int(r.cache.status.item()) == 0


def test_other_stream_and_graph(kv8):
    """A step captured on its own stream and replayed, each replay a new step:
    lengths, rows and table are read when the graph runs.  Two graphs share
    one workspace."""
    r = Run(kv8, 2, 2, 2, 128, 32, "int8", "bfloat16", 100)
    r.append([30, 62])
    x = torch.zeros((2, 4 + 4, 128), dtype=torch.bfloat16, device="cuda")
    q_out, out = torch.zeros_like(x[:, :4]).contiguous(), torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda")
    ws = kv8.alloc_workspace(r.cache, 4, 1)
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            r.cache.seq_len += 1
            kv8.kv8_append(r.cache, x[:, 4:6], x[:, 6:], q=x[:, :4], q_out=q_out, rope=r.rope)
            kv8.kv8_attn(r.cache, q_out, out, ws, 100)
        graphs.append(g)
    for step in range(6):
        host = r.numbers((2, 8, 128))
        x.copy_(_dev(host, r.dtype))
        graphs[step % 2].replay()
        torch.cuda.synchronize()
        r.q, r.q_out = r.orc.append(host[:, 4:6], host[:, 6:], [0, 1, 2], r.table, False, host[:, :4]), q_out
        r.check_state()
        r.close(_host(out), *r.orc.attention(r.q, [0, 1, 2]))
    # eager on a stream of its own
    with torch.cuda.stream(side):
        o2 = torch.zeros_like(out)
        side.wait_stream(torch.cuda.default_stream())
        kv8.kv8_attn(r.cache, q_out, o2, ws, 100, stream=side)
    side.synchronize()
    assert torch.equal(o2, out)


def test_first_calls_of_a_process_are_captured(kv8):
    """Nothing has to run before a capture: append and attention, both kernels,
    as a new process's first calls."""
    code = """
import torch
from bit_kv_cache_02_gb300 import kv8
c = kv8.KV8Cache(2, 2, 600, 18, head_dim=128, block=64, fmt="e4m3", dtype=torch.bfloat16)
c.block_table.copy_(torch.arange(18).view(2, 9))
x = torch.randn(301, 8, 128, device="cuda").bfloat16()
q, out, eager = (torch.zeros(301, 4, 128, device="cuda", dtype=torch.bfloat16) for _ in range(3))
start = torch.tensor([0, 300, 301], dtype=torch.int32, device="cuda")
ws, rope = kv8.alloc_workspace(c, 4, 300), kv8.rope_table(600, 128)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    c.seq_len += start[1:] - start[:-1]
    kv8.kv8_append(c, x[:, 4:6], x[:, 6:], row_start=start, max_new=300, q=x[:, :4], q_out=q, rope=rope)
    kv8.kv8_attn(c, q, out, ws, 600, row_start=start, max_new=300)
g.replay()
kv8.kv8_attn(c, q, eager, ws, 600, row_start=start, max_new=300)
torch.cuda.synchronize()
assert c.seq_len.tolist() == [300, 1] and int(c.status.item()) == 0
assert torch.equal(out, eager) and bool((out != 0).any(-1).all())
print("captured first")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]


def test_serving_loop(kv8):
    """Prompts, decode steps, draft checking with tokens taken back, a second
    prompt's chunk among decoding sequences: the calls as a server makes them."""
    r = Run(kv8, 4, 2, 4, 128, 64, "e4m3", "bfloat16", 500, seed=11)
    ws = kv8.alloc_workspace(r.cache, 8, 300)
    for new in ([100, 0, 37, 1], [1, 0, 1, 1], [5, 0, 5, 5]):
        r.append(new)
        r.attend(ws=ws)
    # two of the five drafts are rejected: the lengths shrink within the block
    keep = [3 if (n % 64) >= 2 else 5 for n in r.orc.lengths()]
    for s in (0, 2, 3):
        drop = 5 - keep[s]
        r.orc.k[s], r.orc.v[s] = (x[: len(x) - drop] for x in (r.orc.k[s], r.orc.v[s]))
        r.cache.seq_len[s] -= drop
    for new in ([1, 300, 1, 1], [1, 130, 1, 1], [1, 1, 1, 1]):
        r.append(new)
        r.check_state()
        r.attend(ws=ws)
    assert int(r.cache.status.item()) == 0
