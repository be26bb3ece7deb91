"""Cross attention and attention behind shared prefixes with row ranges and groups
that are invalid, over many row tiles: what is invalid sets a status bit, its
rows are left alone, and the workspace serves the next call as before."""

import numpy as np
import pytest
import torch

from test_gpu_kv8 import kv8  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
COUNTERS = 6656  # bytes of merge counters at a workspace's start


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Filled:
    """A cache of random codes, `lens` tokens in each sequence, and queries."""

    def __init__(self, kv8, lens, H, g, rows, D=64, B=64, seed=0):
        self.kv8, self.lens, self.Hq, self.rows = kv8, list(lens), H * g, rows
        self.capacity = -(-max(lens) // B) * B
        gen = torch.Generator(device="cuda").manual_seed(seed)
        nb = self.capacity // B
        self.cache = kv8.KV8Cache(len(lens), H, self.capacity, len(lens) * nb, head_dim=D, block=B,
                                  status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        order = torch.randperm(len(lens) * nb, generator=gen, device="cuda")
        self.cache.block_table.copy_(order.view(len(lens), nb).int())
        self.cache.codes.view(torch.uint8).random_(0, 256, generator=gen)
        self.cache.codes.clamp_min_(-127)
        self.cache.scales.fill_(0.01)
        for w in (self.cache.k_win, self.cache.v_win):
            w.normal_(generator=gen)
        self.cache.seq_len.copy_(_i32(lens))
        self.q = torch.randn((rows, self.Hq, D), generator=gen, device="cuda").half()

    def call(self, which, ws, start, most, groups=None, prefix=None, group_rows=None):
        """(outputs, where 3.0 was not written; status)"""
        self.cache.status.zero_()
        out = torch.full_like(self.q, 3.0)
        if which == "cross":
            self.kv8.kv8_cross_attn(self.cache, self.q, out, ws, self.capacity, row_start=_i32(start), max_rows=most)
        else:
            self.kv8.kv8_shared_attn(self.cache, self.q, out, ws, self.capacity, _i32(groups), _i32(prefix), group_rows,
                                     row_start=_i32(start), max_new=most)
        torch.cuda.synchronize()
        assert int(ws[:COUNTERS].view(torch.int32).abs().sum()) == 0, "counters that stay set"
        return out, int(self.cache.status.item())


@pytest.mark.parametrize("lens,H,falling", [
    ([500, 2000, 3500], 8, [0, 150, 50, 400]),
    ([5685, 3812, 1188, 4962, 431, 1071], 4, [0, 164, 403, 1118, 724, 977, 1283]),
    ([6400, 6100, 8000, 500, 7700, 760, 5000], 8, [0, 383, 88, 449, 520, 110, 167, 533]),
])
def test_cross_row_starts_that_fall(kv8, lens, H, falling):
    """No row of a sequence with many rows is written, those of few are right, and
    calls on the same workspace go on as before."""
    S, rows, most = len(lens), max(falling), 1000
    r = Filled(kv8, lens, H, 4, rows)
    ws = kv8.alloc_cross_workspace(r.cache, 4 * H, most)
    rising = [rows * s // S for s in range(S + 1)]
    want, st = r.call("cross", ws, rising, most)
    assert st == 0 and not (want == 3.0).any()
    out, st = r.call("cross", ws, falling, most)
    assert st == 2 and (out == 3.0).all()
    # ten rows of the last sequence beside them: the rows kernel's
    few = falling[:-1] + [falling[-2] + 10]
    out, st = r.call("cross", ws, few, most)
    right, _ = r.call("cross", ws, [0] * (S - 1) + few[-2:], most)
    assert st == 2 and torch.equal(out[few[-2]:few[-1]], right[few[-2]:few[-1]])
    again, st = r.call("cross", ws, rising, most)
    assert st == 0 and torch.equal(again, want)


@pytest.mark.parametrize("H,g,units,falling", [
    (1, 4, [200, 2, 2, 200, 200, 1, 200, 200], [0, 218, 543, 80, 449, 119, 568, 121, 270]),
    (4, 4, [30, 6, 61, 4, 40, 11], [0, 164, 403, 1118, 724, 977, 1283]),
])
def test_shared_bounds_that_fall(kv8, H, g, units, falling):
    """row_start or group_start that falls: the status bit, and the workspace serves
    later calls."""
    S, rows, most = len(units), max(falling), 700
    prefix = [128 * u for u in units]
    r = Filled(kv8, [p + most + 30 for p in prefix], H, g, rows)
    ws = kv8.alloc_shared_workspace(r.cache, H * g, rows, most, rows)
    rising, groups = [rows * s // S for s in range(S + 1)], list(range(S + 1))
    args = dict(groups=groups, prefix=prefix, group_rows=rows)
    want, st = r.call("shared", ws, rising, most, **args)
    assert st == 0 and not (want == 3.0).any()
    rng = np.random.default_rng(1)
    cases = [dict(start=falling)]
    for _ in range(6):
        at = rng.integers(0, rows, S + 1)
        cases.append(dict(start=[0, *sorted(at[1:-1]), rows], groups=[int(x) for x in rng.integers(0, S + 1, S + 1)]))
        cases.append(dict(start=[int(x) for x in at]))
    for kw in cases:
        kw = dict(args, **kw)
        falls = any(y < x for line in (kw["start"], kw["groups"]) for x, y in zip(line, line[1:]))
        out, st = r.call("shared", ws, most=most, **kw)
        assert st & 2 or not falls, kw
        again, st = r.call("shared", ws, rising, most, **args)
        assert st == 0 and torch.equal(again, want), kw


def test_a_shut_out_sequence_does_not_stall_the_call(kv8):
    """A sequence above max_len that shares blocks has its rows taken out of its
    group's join.  That takes no longer than the zeros that it gets anyway: a call
    in which it is of no group takes as long, to within half."""
    n = 2000
    r = Filled(kv8, [300, 9000, 300], 8, 4, n + 2)
    ws = kv8.alloc_shared_workspace(r.cache, 32, n + 2, n, n + 2)
    start, prefix, out = _i32([0, 1, n + 1, n + 2]), _i32([256]), torch.empty_like(r.q)

    def time(groups):
        groups, best = _i32(groups), float("inf")
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):
                kv8.kv8_shared_attn(r.cache, r.q, out, ws, 8000, groups, prefix, n + 2, row_start=start, max_new=n)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    alone = time([0, 1])
    assert time([0, 3]) <= 1.5 * alone
    assert (out[1:n + 1] == 0).all() and (out[[0, n + 1]] != 0).any()


def test_an_invalid_group_s_rows_are_left_alone(kv8):
    """All of them, those of a sequence above max_len too, which gets zeros in a
    valid group."""
    r = Filled(kv8, [300, 900, 310, 400], 2, 4, 8)
    ws = kv8.alloc_shared_workspace(r.cache, 8, 8, 2, 8)
    start = [0, 2, 4, 6, 8]

    def call(prefix, max_len, group_rows=6):
        r.capacity, was = max_len, r.capacity
        out, st = r.call("shared", ws, start, 2, groups=[0, 3], prefix=[prefix], group_rows=group_rows)
        r.capacity = was
        return out, st

    # Other rows are the same within the roundings: without the sequence the work is
    # cut at other places, so that weights are rounded to fp16 relative to other
    # maxima.  Each is off by 2^-11 of itself at most, an output by 2^-11 of the
    # largest value, and by 2^-11 of itself once it is fp16; sums in fp32 of 300
    # tokens by 300 * 2^-24 of that value.  Two of them differ by twice that.
    value = max(1.27, float(r.cache.v_win.abs().max()))  # of blocks: 127 * 0.01
    want, st = call(256, 900)
    assert st == 0

    def same(rows):
        x, y = out[rows].double(), want[rows].double()
        return bool(((x - y).abs() <= 2.0 ** -10 * (value * (1 + 300 * 2.0 ** -13) + y.abs())).all())

    out, st = call(256, 500)
    assert st == 8 and (out[2:4] == 0).all() and same([0, 1, 4, 5, 6, 7])
    for prefix, group_rows in ((-1, 6), (501, 6), (320, 6), (256, 5)):
        out, st = call(prefix, 500, group_rows)
        assert st == 2 and (out[:6] == 3.0).all() and same([6, 7]), (prefix, group_rows)


def test_a_start_far_behind_the_rows(kv8):
    """A row range that ends at 2^31 - 1, whose rows times the queries per KV head
    pass 32 bits, is invalid; the other sequences' rows are what they were."""
    lens, rows = [1200, 3900, 6400, 500], 900
    r = Filled(kv8, lens, 1, 512, rows)
    ws = kv8.alloc_cross_workspace(r.cache, 512, 600)
    want, st = r.call("cross", ws, [0, 300, 900, 900, 900], 600)
    assert st == 0
    out, st = r.call("cross", ws, [0, 300, 900, 2 ** 31 - 1, 2 ** 31 - 1], 600)
    assert st == 2 and torch.equal(out, want)
    ws = kv8.alloc_shared_workspace(r.cache, 512, rows, 600, 900)
    args = dict(groups=[0, 2, 4], prefix=[300, 400], group_rows=900)
    want, st = r.call("shared", ws, [0, 300, 900, 900, 900], 600, **args)
    assert st == 0 and not (want == 3.0).any()
    out, st = r.call("shared", ws, [0, 300, 900, 2 ** 31 - 1, 2 ** 31 - 1], 600, **args)
    assert st == 2 and torch.equal(out, want)
