"""Cases of the 8-bit paged KV cache: appending rotated keys and values, and attention over the cache.

Each case is one call on a cache that holds `ctx` tokens per sequence and gets `new` tokens per sequence:

* "append": rotate queries and keys to their positions, store keys and values; blocks of `block` tokens that
  fill are quantised to 8 bits with one scale for each (block, KV head, keys or values), the rest stays in 16
  bits in a window.
* "attend": attention of the new tokens' queries over the cache, each token up to its own position.

The cache: codes [blocks][kv_heads][2][block][dim] (0: keys, 1: values), scales [blocks][kv_heads][2], a block
table [seqs][max_blocks], and the window [seqs][kv_heads][block][dim] of the last, incomplete block.
"""

import math
import random

import torch

own = False  # whether run() calls the framework's kernels


# ------------------------------------------------------------------ cases

def _case(op, fmt, dtype, seqs, kv_heads, group, ctx, new, singles=0, dim=128, block=64, rot=None, interleaved=False,
          mix=0, name=None):
    c = dict(op=op, fmt=fmt, dtype=dtype, seqs=seqs, kv_heads=kv_heads, group=group, dim=dim, block=block,
             ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=new[0], new_hi=new[1], singles=singles,
             rot=dim if rot is None else rot, interleaved=interleaved, mix=mix)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's next token: a single sequence, nothing but launch latency
        _case("append", "int8", "bfloat16", 1, 8, 4, (700, 700), (1, 1), name="append one token"),
        # a decode step of a full batch: windows at all fill levels, one in `block` of them completes a block
        _case("append", "e4m3", "float16", 64, 8, 4, (1024, 8192), (1, 1), block=32, mix=1, name="append batch step"),
        # prompts of a batch with as many KV heads as query heads
        _case("append", "int8", "float16", 16, 32, 1, (0, 0), (4096, 4096), mix=2, name="append prompts"),
        # chunks of several prompts of uneven length behind stored ones; half the head rotated, neighbours paired
        _case("append", "e4m3", "bfloat16", 7, 4, 6, (1, 3000), (500, 2500), dim=64, block=128, rot=32,
              interleaved=True, mix=3, name="append ragged chunks"),
        # one user's next token on a short context
        _case("attend", "int8", "bfloat16", 1, 8, 4, (300, 300), (1, 1), name="token, short"),
        # a decode step of the multi-head shape that this library's benchmark decodes
        _case("attend", "int8", "float16", 16, 32, 1, (4096, 4096), (1, 1), mix=4, name="token, heads"),
        # a decode step of a large grouped-query batch with uneven contexts
        _case("attend", "e4m3", "bfloat16", 64, 8, 4, (1024, 8192), (1, 1), block=32, mix=5, name="token, ragged"),
        # one very long context; the pool is past 2^31 bytes
        _case("attend", "int8", "float16", 1, 8, 4, (1048576, 1048576), (1, 1), block=128, mix=6, name="token, long"),
        # checking a few draft tokens per sequence
        _case("attend", "e4m3", "float16", 16, 8, 4, (2000, 6000), (3, 8), mix=7, name="verify drafts"),
        # one chunk of a long prompt behind its stored part
        _case("attend", "int8", "bfloat16", 1, 8, 4, (6144, 6144), (2048, 2048), mix=8, name="chunk of a prompt"),
        # whole prompts of uneven length
        _case("attend", "int8", "float16", 4, 32, 1, (0, 0), (1500, 4096), mix=9, name="prompts"),
        # a mixed batch: most sequences decode one token, a few bring a chunk; small heads, odd group
        _case("attend", "e4m3", "bfloat16", 24, 4, 7, (200, 4000), (256, 1000), singles=20, dim=64, block=32, mix=10,
              name="mixed batch"),
    ]


def _span(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    top = [(work(c), _padded(c)) for c in listed()]
    while True:
        op = rng.choice(["append", "attend", "attend"])
        dim, block = rng.choice([64, 128, 128]), rng.choice([32, 64, 128])
        kv_heads, group = rng.choice([1, 2, 3, 4, 8, 8, 16, 32]), rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 12, 16])
        seqs = _span(rng, 1, 96)
        ctx_hi = _span(rng, 1, 65536)
        ctx_lo = rng.randint(0, ctx_hi) if rng.random() < 0.7 else ctx_hi
        new_hi = 1 if rng.random() < 0.4 else _span(rng, 2, 4096)
        new_lo = rng.randint(1, new_hi)
        singles = rng.randint(0, seqs - 1) if new_hi > 1 and rng.random() < 0.3 else 0
        c = _case(op, rng.choice(["int8", "e4m3"]), rng.choice(["float16", "bfloat16"]), seqs, kv_heads, group,
                  (ctx_lo, ctx_hi), (new_lo, new_hi), singles, dim, block, rng.choice([0, 32, dim, dim]),
                  rng.random() < 0.3, rng.randrange(1 << 20))
        w, p = work(c), _padded(c)
        if any(w["bytes"] <= t["bytes"] and w["flops"] <= t["flops"] and p <= q for t, q in top) \
                and w["bytes"] < 1e9 and p < 4e9:
            return c


def _lengths(c):
    """Tokens stored before the call and tokens of the call, for each sequence."""
    rng = random.Random(1000003 * c["mix"] + c["seqs"])
    ctx = [rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["seqs"])]
    new = [1 if s < c["singles"] else rng.randint(c["new_lo"], c["new_hi"]) for s in range(c["seqs"])]
    order = list(range(c["seqs"]))
    rng.shuffle(order)
    return ctx, [new[i] for i in order]


def _padded(c):
    """Values of the plain form's largest tensor."""
    ctx, new = _lengths(c)
    most = max(x + n for x, n in zip(ctx, new)) + c["block"]
    heads = c["kv_heads"] * c["seqs"]
    return heads * most * max(c["dim"], c["group"] * max(new) if c["op"] == "attend" else 0)


def work(c):
    ctx, new = _lengths(c)
    d, hk, b = c["dim"], c["kv_heads"], c["block"]
    hq = hk * c["group"]
    rows = sum(new)
    if c["op"] == "append":
        full = sum((x + n) // b - x // b for x, n in zip(ctx, new))  # blocks that the call completes
        old = sum(x % b for x, n in zip(ctx, new) if (x + n) // b > x // b)  # window tokens that go into them
        kept = sum((x + n) % b if (x + n) // b > x // b else n for x, n in zip(ctx, new))
        read = 2 * d * rows * (hq + 2 * hk) + 4 * d * hk * old + 4 * c["rot"] * rows
        written = 2 * d * rows * hq + 2 * hk * full * (b * d + 4) + 4 * d * hk * kept
        return {"bytes": read + written, "flops": 3 * c["rot"] * rows * (hq + hk) + 4 * d * hk * b * full}
    full = sum((x + n) // b for x, n in zip(ctx, new))
    tail = sum((x + n) % b for x, n in zip(ctx, new))
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


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ctx, new = _lengths(c)
    s, hk, b, d = c["seqs"], c["kv_heads"], c["block"], c["dim"]
    hq = hk * c["group"]
    dtype = getattr(torch, c["dtype"])
    lens = [x + n for x, n in zip(ctx, new)]
    capacity = -(-max(lens) // b) * b
    stored = ctx if c["op"] == "append" else lens  # tokens in the cache before the call
    need = [x // b for x in lens]
    nb = max(1, sum(need))
    order = torch.randperm(nb, generator=gen, device="cuda").int()
    table = torch.full((s, capacity // b), -1, dtype=torch.int32, device="cuda")
    seq_of = torch.tensor([i for i in range(s) for _ in range(need[i])], device="cuda", dtype=torch.long)
    idx_of = torch.tensor([j for i in range(s) for j in range(need[i])], device="cuda", dtype=torch.long)
    table[seq_of, idx_of] = order[: sum(need)]
    code_type = torch.int8 if c["fmt"] == "int8" else torch.float8_e4m3fn
    codes = torch.zeros((nb, hk, 2, b, d), dtype=code_type, device="cuda")
    scales = torch.zeros((nb, hk, 2), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (hk * b * d))
    for lo in range(0, nb, step):  # the stored blocks hold tokens like any others
        n = min(step, nb - lo)
        for j in (0, 1):
            codes[lo:lo + n, :, j], scales[lo:lo + n, :, j] = _quantised(
                _tokens((n, hk, b, d), dtype, gen, j == 0), c["fmt"])
    win = [_tokens((s, hk, b, d), dtype, gen, j == 0) for j in (0, 1)]
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    rows = start[-1]
    state = dict(c, codes=codes, scales=scales, k_win=win[0], v_win=win[1], table=table, ctx=ctx, new=new,
                 capacity=capacity, max_new=max(new), max_len=max(lens), num_q_heads=hq,
                 seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 row_start=torch.tensor(start, dtype=torch.int32, device="cuda"))
    if c["op"] == "append":
        # queries, keys and values as one projection leaves them
        qkv = torch.randn((rows, hq + 2 * hk, d), generator=gen, device="cuda")
        qkv[:, hq:hq + hk, :: d // 4] *= 6
        qkv = qkv.to(dtype)
        state.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:],
                     q_out=torch.empty((rows, hq, d), dtype=dtype, device="cuda"))
        if c["rot"]:
            ang = torch.arange(capacity, device="cuda", dtype=torch.float64)[:, None] * \
                10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
            state["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    else:
        state.update(q=_tokens((rows, hq, d), dtype, gen, False),
                     out=torch.empty((rows, hq, d), dtype=dtype, device="cuda"))
    # where the plain form finds each row, and which blocks this call completes
    state["row_seq"] = torch.tensor([i for i in range(s) for _ in range(new[i])], device="cuda")
    state["row_pos"] = torch.tensor([x + t for x, n in zip(ctx, new) for t in range(n)], device="cuda")
    state["done_seq"] = torch.tensor([i for i in range(s) for _ in range(ctx[i] // b, lens[i] // b)],
                                     device="cuda", dtype=torch.long)
    state["done_idx"] = torch.tensor([j for i in range(s) for j in range(ctx[i] // b, lens[i] // b)],
                                     device="cuda", dtype=torch.long)
    assert all(x <= y for x, y in zip(stored, lens))
    return state


# -------------------------------------------------------------- plain form

def _rotated(x, st, cos_sin):
    """[rows, heads, dim] with the first `rot` channels of each head rotated to the rows' positions."""
    r = st["rot"]
    if not r:
        return x.clone()
    cos, sin = cos_sin[:, None, : r // 2], cos_sin[:, None, r // 2:]
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
    at = st["rope"][st["row_pos"]] if st["rot"] else None
    st["q_out"].copy_(_rotated(st["q"], st, at))
    ds, di = st["done_seq"], st["done_idx"]
    lens, start = st["seq_len"].long(), st["row_start"].long()
    before = lens - (start[1:] - start[:-1])
    pos = di[:, None] * b + torch.arange(b, device="cuda")  # [done, block]
    fresh = pos >= before[ds][:, None]
    row = torch.where(fresh, start[ds][:, None] + pos - before[ds][:, None], 0)
    kept = st["row_pos"] >= (lens // b * b)[st["row_seq"]]  # rows that stay in the window
    for j, (x, win) in enumerate(((_rotated(st["k"], st, at), st["k_win"]), (st["v"], st["v_win"]))):
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
        x = st["codes"][:, :, j].float() if st["fmt"] == "int8" else st["codes"][:, :, j].to(torch.float32)
        x = (x * st["scales"][:, :, j, None, None])[table]  # [seqs, nb, heads, block, dim]
        x[at, lens // b] = win.float()
        kv.append(x.transpose(1, 2).reshape(s, hk, nb * b, d))
    n = st["max_new"]
    inside = st["row_pos"] - (lens - (start[1:] - start[:-1]))[st["row_seq"]]
    q = torch.zeros((s, n, hk * g, d), device="cuda")
    q[st["row_seq"], inside] = st["q"].float()
    q = q.view(s, n, hk, g, d).permute(0, 2, 3, 1, 4).reshape(s, hk, g * n, d)
    z = q @ kv[0].transpose(2, 3)
    z = z.mul_(1 / math.sqrt(d)).view(s, hk, g, n, nb * b)
    p = torch.arange(nb * b, device="cuda")
    last = (lens - (start[1:] - start[:-1]))[:, None] + torch.arange(n, device="cuda")  # each row's own position
    hidden = p > torch.minimum(last, lens[:, None] - 1)[..., None]
    z.masked_fill_(hidden[:, None, None], -math.inf)
    z -= z.amax(-1, keepdim=True)
    z.exp_()
    z /= z.sum(-1, keepdim=True)
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
        st["cache"] = kv8.KV8Cache(st["seqs"], st["kv_heads"], st["capacity"], st["codes"].shape[0],
                                   head_dim=st["dim"], block=st["block"], fmt=st["fmt"],
                                   dtype=getattr(torch, st["dtype"]), codes=st["codes"], scales=st["scales"],
                                   k_win=st["k_win"], v_win=st["v_win"], seq_len=st["seq_len"],
                                   block_table=st["table"])
        if st["op"] == "attend":
            st["workspace"] = kv8.alloc_workspace(st["cache"], st["num_q_heads"], st["max_new"])
        st["kv8"] = kv8
    return st["kv8"], st["cache"]


def run(st):
    if not own:
        return _append_plain(st) if st["op"] == "append" else _attend_plain(st)
    kv8, cache = _handle(st)
    if st["op"] == "append":
        kv8.kv8_append(cache, st["k"], st["v"], row_start=st["row_start"], max_new=st["max_new"], q=st["q"],
                       q_out=st["q_out"], rope=st.get("rope"), interleaved=st["interleaved"])
        return _append_outputs(st)
    kv8.kv8_attn(cache, st["q"], st["out"], st["workspace"], st["max_len"], row_start=st["row_start"],
                 max_new=st["max_new"])
    return st["out"]


# ----------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_attend(st, work(case)["flops"])


def _turned(x, tab, r, interleaved):
    """The rotation's definition: products and sums in 32 bits, one after the other, then 16 bits."""
    def fl(v):
        return v.float().double()
    if not r:
        return x
    y, half = x.clone(), r // 2
    first = range(0, r, 2) if interleaved else range(half)
    for i, ch in enumerate(first):
        other = ch + 1 if interleaved else ch + half
        cs, sn = tab[:, i].double()[:, None], tab[:, half + i].double()[:, None]
        a, b = x[..., ch].double(), x[..., other].double()
        y[..., ch] = fl(fl(a * cs) - fl(b * sn)).to(x.dtype)
        y[..., other] = fl(fl(b * cs) + fl(a * sn)).to(x.dtype)
    return y


def _exact_append(st):
    b, dtype = st["block"], st["q"].dtype
    tab = st["rope"][st["row_pos"]] if st["rot"] else None
    k, v = _turned(st["k"], tab, st["rot"], st["interleaved"]), st["v"]
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
    return {"q": _turned(st["q"], tab, st["rot"], st["interleaved"]).double(),
            "codes": codes if st["fmt"] != "int8" else codes.to(torch.int8), "scales": scales,
            "k_win": wins[0].double(), "v_win": wins[1].double()}


def _exact_attend(st, flops):
    if flops > 3e12:
        return None
    b, d, g = st["block"], st["dim"], st["group"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for s, (old, n) in enumerate(zip(st["ctx"], st["new"])):
        total = old + n
        full = total // b
        blk = st["table"][s, :full].long()
        for h in range(st["kv_heads"]):
            k, v = (torch.cat([(st["codes"][blk, h, j].to(torch.float32).double()
                                * st["scales"][blk, h, j].double()[:, None, None]).reshape(full * b, d),
                               w[s, h, : total - full * b].double()])
                    for j, w in ((0, st["k_win"]), (1, st["v_win"])))
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                q = st["q"][at + i:at + i + m, h * g:(h + 1) * g].double()
                w = torch.einsum("ngd,pd->gnp", q, k) / d ** 0.5
                far = torch.arange(total, device="cuda")[None] > (old + i + torch.arange(m, device="cuda"))[:, None]
                w = torch.softmax(w.masked_fill(far, float("-inf")), -1)
                out[at + i:at + i + m, h * g:(h + 1) * g] = torch.einsum("gnp,pd->ngd", w, v)
        at += n
    return out
