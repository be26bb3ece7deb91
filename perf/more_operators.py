"""Cases of the 8-bit paged KV cache beyond one causal sequence: positions with several axes, attention to an
encoder's states, and attention of sequences that share a prefix.

Each case is one call:

* "axes": append of new tokens whose positions have several axes (time, height and width of image patches, say);
  each pair of channels turns by one of them.  Blocks of `block` tokens that fill are quantised to 8 bits with one
  scale for each (block, KV head, keys or values), the rest stays in 16 bits in a window.
* "cross": attention of a decoder's rows (tokens, or beams, or both) to all tokens of an encoder's states.
* "shared": causal attention of sequences of which groups share their first tokens, in the same blocks.

The cache: codes [blocks][kv_heads][2][block][dim] (0: keys, 1: values), scales [blocks][kv_heads][2], a block
table [seqs][max_blocks], and the window [seqs][kv_heads][block][dim] of the last, incomplete block.
"""

import math
import random

import torch

own = False  # whether run() calls the framework's kernels


# ------------------------------------------------------------------ cases

def _case(op, fmt, dtype, kv_heads, group, dim=128, block=64, mix=0, name=None, **sizes):
    c = dict(op=op, fmt=fmt, dtype=dtype, kv_heads=kv_heads, group=group, dim=dim, block=block, mix=mix, **sizes)
    return dict(c, name=name) if name else c


def _axes(fmt, dtype, seqs, kv_heads, group, ctx, new, axes, cyclic=False, rot=None, interleaved=False, dim=128, **more):
    return _case("axes", fmt, dtype, kv_heads, group, dim=dim, seqs=seqs, ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=new[0],
                 new_hi=new[1], axes=axes, cyclic=cyclic, rot=dim if rot is None else rot, interleaved=interleaved,
                 **more)


def _cross(fmt, dtype, seqs, kv_heads, group, ctx, rows, **more):
    return _case("cross", fmt, dtype, kv_heads, group, seqs=seqs, ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=rows[0],
                 new_hi=rows[1], **more)


def _shared(fmt, dtype, groups, members, kv_heads, group, prefix, ctx, new, **more):
    return _case("shared", fmt, dtype, kv_heads, group, groups=groups, mem_lo=members[0], mem_hi=members[1],
                 pre_lo=prefix[0], pre_hi=prefix[1], ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=new[0], new_hi=new[1], **more)


def listed():
    return [
        # one user's next token behind a prompt with an image: nothing but launch latency
        _axes("int8", "bfloat16", 1, 8, 4, (700, 700), (1, 1), 3, name="axes, one token"),
        # a decode step of a full batch; the pairs take the three axes in turn
        _axes("e4m3", "float16", 64, 8, 4, (1024, 8192), (1, 1), 3, cyclic=True, block=32, mix=1,
              name="axes, batch step"),
        # prompts of text and images
        _axes("int8", "bfloat16", 16, 8, 4, (0, 0), (1000, 4096), 3, mix=2, name="axes, prompts"),
        # patches of several images (rows and columns), half the head rotated, neighbours paired
        _axes("e4m3", "bfloat16", 7, 4, 6, (1, 2000), (500, 2500), 2, rot=32, interleaved=True, dim=64, block=128,
              mix=3, name="axes, ragged patches"),
        # one user's next token over a short text's states
        _cross("int8", "bfloat16", 1, 8, 4, (300, 300), (1, 1), name="cross, token"),
        # beam search over the states of pieces of sound: four beams read the same ones
        _cross("int8", "float16", 16, 16, 1, (1500, 1500), (4, 4), dim=64, block=32, mix=4, name="cross, beams"),
        # a decode step of a batch over images of different sizes
        _cross("e4m3", "bfloat16", 48, 8, 4, (576, 6400), (1, 1), mix=5, name="cross, batch"),
        # the given starts of the outputs, many rows at once, as a scorer of transcripts runs them
        _cross("int8", "float16", 16, 16, 1, (1500, 1500), (200, 448), dim=64, mix=6, name="cross, prompts"),
        # four answers to one short prompt: latency
        _shared("int8", "bfloat16", 1, (4, 4), 8, 4, (512, 512), (1, 40), (1, 1), name="shared, few"),
        # a decode step of a batch behind one long system prompt
        _shared("e4m3", "bfloat16", 1, (64, 64), 8, 4, (4096, 4096), (64, 1024), (1, 1), block=32, mix=7,
                name="shared, batch"),
        # several prompts with some answers each, a few draft tokens at a time; small heads, odd group
        _shared("e4m3", "float16", 12, (1, 8), 4, 7, (1000, 6000), (1, 500), (1, 5), dim=64, block=128, mix=8,
                name="shared, groups"),
        # questions about one long document, appended as chunks
        _shared("int8", "bfloat16", 1, (6, 6), 8, 4, (8192, 8192), (0, 0), (100, 500), mix=9,
                name="shared, questions"),
    ]


def _span(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    top = [(work(c), _padded(c)) for c in listed()]
    while True:
        op = rng.choice(["axes", "cross", "shared"])
        dim, block = rng.choice([64, 128, 128]), rng.choice([32, 64, 128])
        heads = (rng.choice([1, 2, 3, 4, 8, 8, 16, 20]), rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 12, 16]))
        types = (rng.choice(["int8", "e4m3"]), rng.choice(["float16", "bfloat16"]))
        new_hi = 1 if rng.random() < 0.4 else _span(rng, 2, 2048)
        new = (rng.randint(1, new_hi), new_hi)
        more = dict(dim=dim, block=block, mix=rng.randrange(1 << 20))
        if op == "axes":
            ctx_hi = _span(rng, 1, 32768)
            rot = rng.choice([16, 32, 48, dim, dim])
            c = _axes(*types, _span(rng, 1, 96), *heads, (rng.randint(0, ctx_hi), ctx_hi), new, rng.randint(1, 4),
                      cyclic=rng.random() < 0.4, rot=rot, interleaved=rng.random() < 0.3, **more)
        elif op == "cross":
            ctx_hi = _span(rng, 1, 32768)
            c = _cross(*types, _span(rng, 1, 96), *heads, (rng.randint(0, ctx_hi), ctx_hi), new, **more)
        else:
            mem_hi, pre_hi, ctx_hi = _span(rng, 1, 48), _span(rng, 1, 16384), _span(rng, 1, 4096)
            c = _shared(*types, _span(rng, 1, 16), (rng.randint(1, mem_hi), mem_hi), *heads,
                        (rng.randint(0, pre_hi), pre_hi), (rng.randint(0, ctx_hi), ctx_hi), new, **more)
        w, p = work(c), _padded(c)
        if any(w["bytes"] <= t["bytes"] and w["flops"] <= t["flops"] and p <= q for t, q in top) \
                and w["bytes"] < 1e9 and p < 4e9:
            return c


def _plan(c):
    """For each sequence: tokens stored before the call, tokens (rows) of the call, its group; for each group: the
    tokens that its sequences share."""
    rng = random.Random(1000003 * c["mix"] + c["kv_heads"])
    if c["op"] != "shared":
        ctx = [rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["seqs"])]
        return ctx, [rng.randint(c["new_lo"], c["new_hi"]) for _ in ctx], [0] * len(ctx), []
    ctx, new, of, prefix = [], [], [], []
    for g in range(c["groups"]):
        prefix.append(rng.randint(c["pre_lo"], c["pre_hi"]))
        for _ in range(rng.randint(c["mem_lo"], c["mem_hi"])):
            ctx.append(prefix[g] + rng.randint(c["ctx_lo"], c["ctx_hi"]))
            new.append(rng.randint(c["new_lo"], c["new_hi"]))
            of.append(g)
    return ctx, new, of, prefix


def _lengths(c):
    """Tokens of each sequence in the cache once the call's own are in it."""
    ctx, new, _, _ = _plan(c)
    return ctx if c["op"] == "cross" else [x + n for x, n in zip(ctx, new)]


def _padded(c):
    """Values of the plain form's largest tensor."""
    _, new, _, _ = _plan(c)
    lens = _lengths(c)
    most = max(lens) + c["block"]
    return c["kv_heads"] * len(lens) * most * max(c["dim"], c["group"] * max(new) if c["op"] != "axes" else 0)


def _table_rows(c):
    # one axis: positions of tokens from a text of which the cache holds a part
    return max(_lengths(c)) * (2 if c["axes"] == 1 else 1)


def work(c):
    ctx, new, of, prefix = _plan(c)
    d, hk, b = c["dim"], c["kv_heads"], c["block"]
    hq = hk * c["group"]
    rows = sum(new)
    if c["op"] == "axes":
        full = sum((x + n) // b - x // b for x, n in zip(ctx, new))  # blocks that the call completes
        old = sum(x % b for x, n in zip(ctx, new) if (x + n) // b > x // b)  # window tokens that go into them
        kept = sum((x + n) % b if (x + n) // b > x // b else n for x, n in zip(ctx, new))
        angles = 4 * c["rot"] * min(rows * c["axes"], _table_rows(c))
        read = 2 * d * rows * (hq + 2 * hk) + 4 * d * hk * old + angles + 4 * c["axes"] * rows
        written = 2 * d * rows * hq + 2 * hk * full * (b * d + 4) + 4 * d * hk * kept
        return {"bytes": read + written, "flops": 3 * c["rot"] * rows * (hq + hk) + 4 * d * hk * b * full}
    lens = _lengths(c)
    full = sum(x // b for x in lens)
    tail = sum(x % b for x in lens)
    if c["op"] == "cross":
        seen = sum(n * x for x, n in zip(lens, new))
    else:
        full -= sum((of.count(g) - 1) * (p // b) for g, p in enumerate(prefix))
        seen = sum(n * x + n * (n + 1) // 2 for x, n in zip(ctx, new))  # visible (row, key) pairs
    return {"bytes": hk * (full * (2 * b * d + 8) + 4 * d * tail) + 4 * d * rows * hq, "flops": 4 * d * hq * seen}


# ----------------------------------------------------------------- inputs

def _tokens(shape, dtype, gen, keys):
    """Normal values; keys with a few large channels, as real keys have."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if keys:
        x[..., :: shape[-1] // 4] *= 6
    return x.to(dtype)


def _quantised(x, fmt):
    """[..., block, dim] in 16 bits -> (codes, scale [...]): one scale for each block."""
    amax = x.float().abs().amax((-1, -2)).clamp_min(2.0 ** -100).double()
    if fmt == "int8":
        scale, inv = (amax / 127).float(), (127 / amax).float()
        codes = (x.double() * inv.double()[..., None, None]).round().to(torch.int8)
    else:
        m, e = torch.frexp(amax)  # the smallest power of two that brings amax to 448 or less
        k = e - 9 + (m > 0.875)
        scale = torch.ldexp(torch.ones_like(amax), k).float()
        codes = (x.float() / scale[..., None, None]).to(torch.float8_e4m3fn)
    return codes, scale


def _axis_of_pairs(c):
    """The axis that each pair of channels turns by."""
    n, a = c["rot"] // 2, c["axes"]
    if c["cyclic"]:
        return [i % a for i in range(n)]
    first = n // 4 if a == 3 else n // a  # time gets a quarter of the pairs, height and width share the rest
    sizes = [first] + [(n - first) // (a - 1)] * (a - 1) if a > 1 else [n]
    sizes[-1] = n - sum(sizes[:-1])
    return [j for j, size in enumerate(sizes) for _ in range(size)]


def _positions(axes, length, skip, top, rng):
    """Positions [axes][length - skip] of a sequence's last tokens.  One axis: a text of which some tokens have been
    dropped.  Else runs of text, where all axes count on together, and grids of patches, where they count the
    patches' places from the grid's start on."""
    if axes == 1:
        at = rng.randint(0, top - length)
        return torch.arange(at + skip, at + length)[None]
    out, size, start = [], 0, 0
    while size < length:
        n = rng.randint(1, 200)
        out.append((start + torch.arange(n)).expand(axes, n))
        start, size = start + n, size + n
        dims = [rng.randint(1, 3)] * (axes - 2) + [rng.randint(1, 28), rng.randint(1, 28)]
        grid = torch.cartesian_prod(*(torch.arange(x) for x in dims)).T
        out.append(start + grid)
        start, size = start + max(dims), size + grid.shape[1]
    return torch.cat(out, 1)[:, skip:length]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ctx, new, of, prefix = _plan(c)
    hk, b, d, s = c["kv_heads"], c["block"], c["dim"], len(ctx)
    hq = hk * c["group"]
    dtype = getattr(torch, c["dtype"])
    lens = _lengths(c)
    capacity = -(-max(*lens, 1) // b) * b
    # the blocks of each sequence: those that its group shares, then its own
    pool, tables, common = 0, [], []
    for p in prefix:
        common.append(list(range(pool, pool + p // b)))
        pool += p // b
    for i in range(s):
        mine = common[of[i]] if prefix else []
        n = lens[i] // b - len(mine)
        tables.append(mine + list(range(pool, pool + n)))
        pool += n
    nb = max(1, pool)
    order = torch.randperm(nb, generator=gen, device="cuda").int()
    table = torch.full((s, capacity // b), -1, dtype=torch.long)
    for i, line in enumerate(tables):
        table[i, : len(line)] = torch.tensor(line, dtype=torch.long)
    table = table.cuda()
    table = torch.where(table >= 0, order[table.clamp_min(0)], -1).int()
    code_type = torch.int8 if c["fmt"] == "int8" else torch.float8_e4m3fn
    codes = torch.zeros((nb, hk, 2, b, d), dtype=code_type, device="cuda")
    scales = torch.zeros((nb, hk, 2), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (hk * b * d))
    for lo in range(0, nb, step):
        n = min(step, nb - lo)
        for j in (0, 1):
            codes[lo:lo + n, :, j], scales[lo:lo + n, :, j] = _quantised(
                _tokens((n, hk, b, d), dtype, gen, j == 0), c["fmt"])
    win = [_tokens((s, hk, b, d), dtype, gen, j == 0) for j in (0, 1)]
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    rows = start[-1]
    state = dict(c, seqs=s, codes=codes, scales=scales, k_win=win[0], v_win=win[1], table=table, ctx=ctx, new=new,
                 lens=lens, capacity=capacity, max_new=max(new), max_len=max(*lens, 1), num_q_heads=hq,
                 seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 row_start=torch.tensor(start, dtype=torch.int32, device="cuda"))
    if c["op"] == "axes":
        # queries, keys and values as one projection leaves them
        qkv = torch.randn((rows, hq + 2 * hk, d), generator=gen, device="cuda")
        qkv[:, hq:hq + hk, :: d // 4] *= 6
        qkv = qkv.to(dtype)
        top, rng = _table_rows(c), random.Random(seed)
        pos = torch.cat([_positions(c["axes"], x, y, top, rng) for x, y in zip(lens, ctx)], 1)
        ang = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
        state.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:],
                     q_out=torch.empty((rows, hq, d), dtype=dtype, device="cuda"),
                     positions=pos.int().cuda(), axis_of=_axis_of_pairs(c),
                     rope=torch.cat([ang.cos(), ang.sin()], 1).float())
    else:
        state.update(q=_tokens((rows, hq, d), dtype, gen, False),
                     out=torch.empty((rows, hq, d), dtype=dtype, device="cuda"))
    if prefix:
        bounds = [of.index(g) for g in range(len(prefix))] + [s]
        state.update(group_start=torch.tensor(bounds, dtype=torch.int32, device="cuda"),
                     prefix_len=torch.tensor(prefix, dtype=torch.int32, device="cuda"),
                     max_group_rows=max(start[y] - start[x] for x, y in zip(bounds, bounds[1:])))
    # where the plain form finds each row, and which blocks this call completes
    state["row_seq"] = torch.tensor([i for i in range(s) for _ in range(new[i])], device="cuda")
    state["row_pos"] = torch.tensor([x + t for x, n in zip(ctx, new) for t in range(n)], device="cuda")
    state["done_seq"] = torch.tensor([i for i in range(s) for _ in range(ctx[i] // b, lens[i] // b)],
                                     device="cuda", dtype=torch.long)
    state["done_idx"] = torch.tensor([j for i in range(s) for j in range(ctx[i] // b, lens[i] // b)],
                                     device="cuda", dtype=torch.long)
    return state


# -------------------------------------------------------------- plain form

def _angles(st):
    """Cosines and sines [rows][rot / 2] of each row's pairs."""
    half = st["rot"] // 2
    axis = torch.tensor(st["axis_of"], device="cuda")
    at = st["positions"][axis].long().T  # [rows, pairs]: the position that each pair turns by
    pair = torch.arange(half, device="cuda")
    return st["rope"][at, pair], st["rope"][at, half + pair]


def _rotated(x, st, angles):
    """[rows, heads, dim] with the first `rot` channels of each head rotated by the rows' angles."""
    r = st["rot"]
    cos, sin = (t[:, None] for t in angles)
    f = x[..., :r].float()
    a, b = (f[..., 0::2], f[..., 1::2]) if st["interleaved"] else (f[..., : r // 2], f[..., r // 2:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    y = x.clone()
    if st["interleaved"]:
        y[..., 0:r:2], y[..., 1:r:2] = ra.to(x.dtype), rb.to(x.dtype)
    else:
        y[..., : r // 2], y[..., r // 2: r] = ra.to(x.dtype), rb.to(x.dtype)
    return y


def _append_plain(st):
    b = st["block"]
    angles = _angles(st)
    st["q_out"].copy_(_rotated(st["q"], st, angles))
    ds, di = st["done_seq"], st["done_idx"]
    lens, start = st["seq_len"].long(), st["row_start"].long()
    before = lens - (start[1:] - start[:-1])
    slot = di[:, None] * b + torch.arange(b, device="cuda")  # [done, block]
    fresh = slot >= before[ds][:, None]
    row = torch.where(fresh, start[ds][:, None] + slot - before[ds][:, None], 0)
    kept = st["row_pos"] >= (lens // b * b)[st["row_seq"]]  # rows that stay in the window
    for j, (x, win) in enumerate(((_rotated(st["k"], st, angles), st["k_win"]), (st["v"], st["v_win"]))):
        if len(ds):
            tok = torch.where(fresh[..., None, None], x[row], win[ds].transpose(1, 2))  # [done, block, heads, dim]
            codes, scale = _quantised(tok.transpose(1, 2), st["fmt"])
            blk = st["table"][ds, di].long()
            st["codes"].view(torch.uint8)[blk, :, j] = codes.view(torch.uint8)
            st["scales"][blk, :, j] = scale
        win[st["row_seq"][kept], :, st["row_pos"][kept] % b] = x[kept]
    return _append_outputs(st)


def _append_outputs(st):
    # the 8-bit values are returned in units of their scales, which stand beside them
    return {"q": st["q_out"], "codes": st["codes"], "scales": st["scales"], "k_win": st["k_win"], "v_win": st["v_win"]}


def _attend_plain(st):
    s, hk, g, b, d = st["seqs"], st["kv_heads"], st["group"], st["block"], st["dim"]
    lens = st["seq_len"].long()
    start = st["row_start"].long()
    nb = st["max_len"] // b + 1
    table = torch.nn.functional.pad(st["table"].long(), (0, 1))[:, :nb].clamp_min(0)
    at = torch.arange(s, device="cuda")
    kv = []
    for j, win in enumerate((st["k_win"], st["v_win"])):
        x = (st["codes"][:, :, j].to(torch.float32) * st["scales"][:, :, j, None, None])[table]
        x[at, lens // b] = win.float()  # [seqs, nb, heads, block, dim]
        kv.append(x.transpose(1, 2).reshape(s, hk, nb * b, d))
    n = st["max_new"]
    inside = torch.arange(len(st["row_seq"]), device="cuda") - start[st["row_seq"]]
    q = torch.zeros((s, n, hk * g, d), device="cuda")
    q[st["row_seq"], inside] = st["q"].float()
    q = q.view(s, n, hk, g, d).permute(0, 2, 3, 1, 4).reshape(s, hk, g * n, d)
    z = q @ kv[0].transpose(2, 3)
    z = z.mul_(1 / math.sqrt(d)).view(s, hk, g, n, nb * b)
    p = torch.arange(nb * b, device="cuda")
    last = (lens - 1)[:, None].expand(s, n)  # the last token that each row sees
    if st["op"] == "shared":
        last = torch.minimum(last, (lens - (start[1:] - start[:-1]))[:, None] + torch.arange(n, device="cuda"))
    z.masked_fill_((p > last[..., None])[:, None, None], -math.inf)
    z -= z.amax(-1, keepdim=True).clamp_min(-3e38)  # rows that see nothing stay empty
    z.exp_()
    z /= z.sum(-1, keepdim=True).clamp_min(1e-30)
    # values of places behind a sequence's end have no weight, whatever they hold
    kv[1].masked_fill_((p >= lens[:, None])[:, None, :, None], 0)
    o = (z.view(s, hk, g * n, nb * b) @ kv[1]).view(s, hk, g, n, d).permute(0, 3, 1, 2, 4).reshape(s, n, hk * g, d)
    st["out"].copy_(o[st["row_seq"], inside])
    return st["out"]


# --------------------------------------------------------------- the calls

def _handle(st):
    """The cache and the workspace, which a program makes once and keeps."""
    if "cache" not in st:
        from bit_kv_cache_02_gb300 import kv8
        cache = kv8.KV8Cache(st["seqs"], st["kv_heads"], st["capacity"], st["codes"].shape[0], head_dim=st["dim"],
                             block=st["block"], fmt=st["fmt"], dtype=getattr(torch, st["dtype"]), codes=st["codes"],
                             scales=st["scales"], k_win=st["k_win"], v_win=st["v_win"], seq_len=st["seq_len"],
                             block_table=st["table"])
        if st["op"] == "axes":
            st["axes_map"] = kv8.rope_axes(st["axis_of"])
        elif st["op"] == "cross":
            st["workspace"] = kv8.alloc_cross_workspace(cache, st["num_q_heads"], st["max_new"])
        else:
            st["workspace"] = kv8.alloc_shared_workspace(cache, st["num_q_heads"], st["q"].shape[0], st["max_new"],
                                                         st["max_group_rows"])
        st["cache"], st["kv8"] = cache, kv8
    return st["kv8"], st["cache"]


def run(st):
    if not own:
        return _append_plain(st) if st["op"] == "axes" else _attend_plain(st)
    kv8, cache = _handle(st)
    if st["op"] == "axes":
        kv8.kv8_append_axes(cache, st["k"], st["v"], st["positions"], st["axes_map"], st["rope"],
                            row_start=st["row_start"], max_new=st["max_new"], q=st["q"], q_out=st["q_out"],
                            interleaved=st["interleaved"])
        return _append_outputs(st)
    if st["op"] == "cross":
        kv8.kv8_cross_attn(cache, st["q"], st["out"], st["workspace"], st["max_len"], row_start=st["row_start"],
                           max_rows=st["max_new"])
    else:
        kv8.kv8_shared_attn(cache, st["q"], st["out"], st["workspace"], st["max_len"], st["group_start"],
                            st["prefix_len"], st["max_group_rows"], row_start=st["row_start"], max_new=st["max_new"])
    return st["out"]


# ----------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "axes" else _exact_attend(st, work(case)["flops"])


def _turned(x, st):
    """The rotation's definition: products and sums in 32 bits, one after the other, then 16 bits."""
    def fl(v):
        return v.float().double()
    r, y = st["rot"], x.clone()
    half = r // 2
    for i, axis in enumerate(st["axis_of"]):
        ch, other = (2 * i, 2 * i + 1) if st["interleaved"] else (i, i + half)
        at = st["positions"][axis].long()
        cs, sn = st["rope"][at, i].double()[:, None], st["rope"][at, half + i].double()[:, None]
        a, b = x[..., ch].double(), x[..., other].double()
        y[..., ch] = fl(fl(a * cs) - fl(b * sn)).to(x.dtype)
        y[..., other] = fl(fl(b * cs) + fl(a * sn)).to(x.dtype)
    return y


def _exact_append(st):
    b, dtype = st["block"], st["q"].dtype
    k, v = _turned(st["k"], st), st["v"]
    codes, scales = st["codes"].to(torch.float32).double(), st["scales"].double()
    wins = [st["k_win"].clone(), st["v_win"].clone()]
    at = 0
    for s, (old, n) in enumerate(zip(st["ctx"], st["new"])):
        first = old // b * b
        for j, x in enumerate((k, v)):
            line = torch.cat([wins[j][s, :, : old - first], x[at:at + n].transpose(0, 1)], 1).double()
            done = line.shape[1] // b
            if done:
                t = line[:, : done * b].reshape(line.shape[0], done, b, -1).transpose(0, 1)
                top = t.abs().flatten(2).amax(2).clamp_min(2.0 ** -100)
                blk = st["table"][s, first // b: first // b + done].long()
                if st["fmt"] == "int8":
                    scales[blk, :, j] = (top / 127).float().double()
                    codes[blk, :, j] = torch.round(t * (127 / top).float().double()[..., None, None])
                else:
                    unit = torch.exp2(torch.ceil(torch.log2(top / 448)))
                    unit = torch.where(top <= 224 * unit, unit / 2, unit)  # where a logarithm was rounded up
                    scales[blk, :, j] = unit
                    y = t / unit[..., None, None]
                    ulp = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
                    codes[blk, :, j] = torch.round(y / ulp) * ulp
            rest = line.shape[1] - done * b
            if done:
                wins[j][s, :, :rest] = line[:, done * b:].to(dtype)
            else:
                wins[j][s, :, old - first: rest] = line[:, old - first:].to(dtype)
        at += n
    return {"q": _turned(st["q"], st).double(), "codes": codes if st["fmt"] != "int8" else codes.to(torch.int8),
            "scales": scales, "k_win": wins[0].double(), "v_win": wins[1].double()}


def _exact_attend(st, flops):
    if flops > 3e12:
        return None
    b, d, g = st["block"], st["dim"], st["group"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for s, (old, n, total) in enumerate(zip(st["ctx"], st["new"], st["lens"])):
        if total == 0:
            out[at:at + n] = 0
        full = total // b
        blk = st["table"][s, :full].long()
        for h in range(st["kv_heads"] if total else 0):
            k, v = (torch.cat([(st["codes"][blk, h, j].to(torch.float32).double()
                                * st["scales"][blk, h, j].double()[:, None, None]).reshape(full * b, d),
                               w[s, h, : total - full * b].double()])
                    for j, w in ((0, st["k_win"]), (1, st["v_win"])))
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                q = st["q"][at + i:at + i + m, h * g:(h + 1) * g].double()
                w = torch.einsum("ngd,pd->gnp", q, k) / d ** 0.5
                if st["op"] == "shared":
                    own_place = old + i + torch.arange(m, device="cuda")
                    w.masked_fill_(torch.arange(total, device="cuda")[None] > own_place[:, None], float("-inf"))
                w = torch.softmax(w, -1)
                out[at + i:at + i + m, h * g:(h + 1) * g] = torch.einsum("gnp,pd->ngd", w, v)
        at += n
    return out
