"""The 8-bit paged cache in plain numpy: what kv8_append and kv8_append_axes
store and what kv8_attn, kv8_cross_attn and kv8_shared_attn return
(include/kv8.h), written from the definitions.

16-bit numbers are carried as float64 arrays that hold representable values.
Every rounding the definition names happens once, at the place it names;
attention is in float64.
"""

from __future__ import annotations

import math

import numpy as np

FLOOR = 2.0 ** -100


def round16(x, dtype):
    """float64 -> nearest float16 or bfloat16 value (ties to even), as float64."""
    x = np.asarray(x, np.float64)
    if dtype == "float16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float64)
    # bfloat16: 8 significant bits, float32's exponents
    out = x.copy()
    fin = np.isfinite(x) & (x != 0)
    m, e = np.frexp(x[fin])
    e = np.maximum(e, -125)  # subnormals share the smallest normal's step
    step = np.ldexp(1.0, e - 8)
    r = np.rint(x[fin] / step) * step
    out[fin] = np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, r), r)
    return out


def round_e4m3(x):
    """float64 -> nearest e4m3 value (ties to even): step 2^(e-3) above 2^-6, 2^-9 below; saturates at 448."""
    x = np.asarray(x, np.float64)
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def rotate(x, table_rows, interleaved, dtype):
    """x [rows, heads, D], table_rows [rows, r] (cosines, then sines): the
    first r channels turned; products and sums rounded to fp32 one by one,
    then the result to 16 bits."""
    r = table_rows.shape[1]
    y = np.array(x, np.float64)
    if r == 0:
        return y
    f32 = np.float32
    i0 = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    i1 = i0 + 1 if interleaved else i0 + r // 2
    a, b = y[..., i0].astype(f32), y[..., i1].astype(f32)
    c, s = table_rows[:, None, : r // 2].astype(f32), table_rows[:, None, r // 2:].astype(f32)
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., i0] = round16(((a * c).astype(f32) - (b * s).astype(f32)).astype(f32), dtype)
        y[..., i1] = round16(((b * c).astype(f32) + (a * s).astype(f32)).astype(f32), dtype)
    return y


def axes_rows(table, positions, axis_of):
    """table [p, r], positions [axes, rows], axis_of: the axis of each of the
    r / 2 pairs -> [rows, r]: the cosines, then the sines, of the rows' pairs;
    NaN where a position is outside the table."""
    half = table.shape[1] // 2
    out = np.full((positions.shape[1], 2 * half), math.nan)
    for i in range(half):
        at = positions[axis_of[i]]
        ok = (at >= 0) & (at < len(table))
        out[ok, i], out[ok, half + i] = table[at[ok], i], table[at[ok], half + i]
    return out


def quantize_block(x, fmt):
    """x [block, D] -> (code values [block, D], fp32 scale as float64)."""
    if not np.isfinite(x).all():
        return np.zeros_like(x), math.nan
    amax = max(float(np.abs(x).max()), FLOOR)
    if fmt == "int8":
        scale, inv = np.float64(np.float32(amax / 127)), np.float64(np.float32(127 / amax))
        return np.rint(x * inv), float(scale)
    k = -400
    while amax > 448 * 2.0 ** k:
        k += 1
    return round_e4m3(x / 2.0 ** k), 2.0 ** k


class OracleKV8:
    """The whole token history of each sequence, from which every state follows."""

    def __init__(self, num_seqs, num_kv_heads, head_dim, block, fmt, dtype):
        self.S, self.H, self.D, self.B, self.fmt, self.dtype = num_seqs, num_kv_heads, head_dim, block, fmt, dtype
        self.k = [np.zeros((0, num_kv_heads, head_dim)) for _ in range(num_seqs)]
        self.v = [np.zeros((0, num_kv_heads, head_dim)) for _ in range(num_seqs)]

    def lengths(self):
        return [len(x) for x in self.k]

    def append(self, k, v, row_start, table=None, interleaved=False, q=None, angles=None):
        """Returns the rotated queries (rows of no sequence as they were).
        angles [rows, r] (axes_rows): the rows' own, whatever their places."""
        q_out = None if q is None else np.array(q, np.float64)
        for s in range(self.S):
            a, b = row_start[s], row_start[s + 1]
            at = np.arange(len(self.k[s]), len(self.k[s]) + b - a)
            rows = angles[a:b] if angles is not None else np.zeros((b - a, 0)) if table is None else table[at]
            self.k[s] = np.concatenate([self.k[s], rotate(k[a:b], rows, interleaved, self.dtype)])
            self.v[s] = np.concatenate([self.v[s], np.array(v[a:b], np.float64)])
            if q is not None:
                q_out[a:b] = rotate(q[a:b], rows, interleaved, self.dtype)
        return q_out

    def block(self, s, b, h, values):
        x = (self.v if values else self.k)[s][b * self.B:(b + 1) * self.B, h]
        assert len(x) == self.B
        return quantize_block(x, self.fmt)

    def stored(self, s, h, values):
        """[L, D]: the tokens as attention sees them."""
        x = (self.v if values else self.k)[s]
        full = len(x) // self.B
        parts = []
        for b in range(full):
            c, scale = self.block(s, b, h, values)
            parts.append(c * scale)
        return np.concatenate(parts + [x[full * self.B:, h]]) if parts else x[:, h]

    def units(self, s, h, rows):
        """For each token the unit of its values in the products with the
        weights, and whether its weight is an fp16 number.  Blocks: their
        scale, 2^-80 where they count as zeros.  The window: fp16 values enter
        as they are.  bf16 values enter, with more than 48 rows per KV head,
        times the power of two that brings the token's largest to [2^14, 2^15)
        (2^81 at most); with fewer as they are, by weights in bf16, and count
        among the others as a block of their size would, from 2^-80 to 1."""
        full = len(self.v[s]) // self.B
        u = [np.zeros(0)]
        for b in range(full):
            scale = self.block(s, b, h, True)[1]
            u.append(np.full(self.B, scale if scale >= 2.0 ** -80 else 2.0 ** -80))
        win = np.abs(self.v[s][full * self.B:, h])
        top = np.where(np.isfinite(win), win, 0).max(1, initial=0)
        e = np.where(top > 0, np.frexp(top)[1], -200)
        if self.dtype == "float16":
            u.append(np.ones(len(win)))
        else:
            u.append(np.ldexp(1.0, np.maximum(e, -66) - 15 if rows > 48 else np.clip(e - 7, -80, 0)))
        in_fp16 = np.ones(len(self.v[s]), bool)
        in_fp16[full * self.B:] = self.dtype == "float16" or rows > 48
        return np.concatenate(u), in_fp16

    def attention(self, q, row_start, softmax_scale=None, causal=True):
        """Each row up to its own position, or (causal False) all tokens.
        q [rows, Hq, D] -> (out, bound): float64 attention, and what the
        kernels' roundings may change it by before the output's own rounding.

        The bound.  A weight is rounded to fp16: 2^-11 of itself, or half a
        step of fp16's subnormals, 2^-25.  Formed is P = w u / U 2^9 or more,
        where u is the unit in which a token's values enter the products (see
        units) and U the largest w u of the row; the sum of P v / u comes back
        times U 2^-9.  A P below 2^-14, that is a w u below 2^-23 U (2^-22 with
        what the scores' errors add), is off by 2^-25, its share of the output
        by 2^-34 U |v| / u.  (It matters where the tokens of large w u have
        small values in a channel, or none: a block of large values of which
        the row sees small ones only counts with its scale.)  A score is a sum of D products accumulated in fp32 (at most
        (D + 16) 2^-24 of the sum of magnitudes, the weight's relative change
        being e^x - 1 < 2 x); adding log2(scale_v) and the reference, both
        below 128 but for the score, rounds four times at 2^-24 * 128: 2^-15.
        The normalizer is a sum of fp32 numbers (2^-24 of itself per term),
        and sums over tokens and partial results are of fp32 too.  All but the
        subnormals' part is relative to sum_p w_p |v_p|.  A bf16 query is
        scaled by a power of two so that its largest element lies in
        [2^14, 2^15) and rounded to fp16: elements that become subnormal are
        off by 2^-25, 2^-39 of the largest; so are the elements of a window
        token, of that token's largest."""
        scale = softmax_scale or 1 / math.sqrt(self.D)
        rows, Hq, _ = q.shape
        g = Hq // self.H
        out, bound = np.zeros(q.shape), np.zeros(q.shape)
        for s in range(self.S):
            a, b = row_start[s], row_start[s + 1]
            n, L = b - a, len(self.k[s])
            if b == a or L == 0:
                continue
            for h in range(self.H):
                K, V = self.stored(s, h, False), self.stored(s, h, True)
                unit, in_fp16 = self.units(s, h, n * g)
                for i in range(n):
                    seen = L - n + i + 1 if causal else L
                    if seen <= 0:
                        continue
                    for j in range(h * g, (h + 1) * g):
                        x = q[a + i, j]
                        with np.errstate(invalid="ignore"):
                            z = K[:seen] @ x * scale
                            mags = np.abs(K[:seen]) @ np.abs(x) * scale
                            if not (np.isfinite(z).all() and np.isfinite(V[:seen]).all()):
                                out[a + i, j] = math.nan
                                continue
                        w = np.exp(z - z.max())
                        w /= w.sum()
                        out[a + i, j] = w @ V[:seen]
                        dz = (self.D + 16) * 2.0 ** -24 * mags.max()
                        if self.dtype == "bfloat16":
                            dz += 2.0 ** -39 * np.abs(x).max() * np.abs(K[:seen]).sum(1).max() * scale
                            dz += 2.0 ** -39 * np.abs(K[:seen]).max() * np.abs(x).sum() * scale
                        rel = 2.0 ** -11 + 2.0 ** -15 + 2 * dz + (2 * seen + 64) * 2.0 ** -24
                        wu = w * unit[:seen]
                        small = in_fp16[:seen] & (wu < 2.0 ** -22 * wu.max())
                        lost = (np.abs(V[:seen][small]) / unit[:seen][small][:, None]).sum(0)
                        bound[a + i, j] = rel * (w @ np.abs(V[:seen])) + 2.0 ** -34 * wu.max() * lost
        return out, bound
