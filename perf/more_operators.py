"""The operators around sparse attention over the paged KV cache: what each
computes, in plain torch, and the cases they are measured at.

  append  pa_rope_and_cache (_fp8, _fp4): new tokens' queries and keys are
          rotated by their positions; rotated queries are written out, rotated
          keys and the values go to their slots of the cache
  bounds  pa_update_key_bounds (_fp8, _fp4): for every block that a call's new
          tokens reach into, each channel's largest and smallest key, in 8 bits
  select  pa_select_blocks: for every query row and KV head, the blocks whose
          bounds promise the largest logits, as a block table of their own
  sparse  pa_decode_sparse (_fp8, _fp4): attention of every row over its own
          blocks
  step    the four in a row: one decode step of a batch

Caches are [num_blocks, num_kv_heads, block_size, head_dim]: 16-bit elements, or
E4M3 codes in uint8 ("fp8"); or FP4 caches ("fp4"), uint8 [num_blocks,
num_kv_heads, block_size * head_dim * 9 / 16], a block and head's bytes being
its tokens' E2M1 codes [block_size, head_dim / 2] (the even element in the low
nibble) and then E4M3 scales, one for 16 elements, [block_size, head_dim / 16].

Rotation.  cos_sin [positions, rotary] holds cosines and then sines, rotary / 2
each, of the angles of a position.  Of the first `rotary` elements of a head, x
and y are elements i and i + rotary / 2 (or, interleaved, 2 i and 2 i + 1):
    x' = x cos_i - y sin_i,    y' = y cos_i + x sin_i
every product and sum rounded to 32 bits and the result to the row's type; the
other elements stay as they are.  FP8 and FP4 caches quantise that result.  A
token with a negative slot is left out altogether.

Bounds of a block and KV head, over the block's tokens below the context's end
(of codes and FP4 scales, without the cache's own scale): with a the largest
magnitude, e the smallest integer (-126 or more) with a <= 127 2^e, and each
channel's extremes hi and lo,  ceil(hi / 2^e), floor(lo / 2^e)  and the scale
2^e; a block of zeros has scale 0 and zeros, one with an infinity or a NaN
scale +inf and zeros.

Selection.  Of a group of query heads sharing a KV head, with a its largest
magnitude and e the smallest integer (-126 or more) with a <= 4095 2^e, every
element becomes c = round(q / 2^e), half to even.  A block's score is its scale
times  sum_d (sum of the group's positive c_d) hi_d + (of the negative) lo_d,
the integer and then the product rounded to 32 bits: 2^-e times a bound on the
sum of the group's logits.  A block of scale +inf has score +inf; a group with
an infinity or a NaN scores zero everywhere else.  A row sees the blocks that
hold its tokens, up to its own position.  Its first `sink` and last `recent`
blocks are always taken, the others by score, ties to the lower index, as many
as `keep` holds, in the order of the sequence.  The table of a row and head
holds their physical blocks (-1 behind them), the length the tokens in them."""
import math

import numpy as np
import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # E2M1 codes 0..7; 8..15 are their negatives


def listed():
    return [
        # append: a step of four short sequences of a small multi-head model
        dict(name="append_tiny", kind="append", tokens=4, hq=4, hkv=4, d=64, bs=16, dtype="fp16",
             kv="16", rotary=64, interleaved=False, far=4096, rows="packed", k_scale=1.0, v_scale=1.0),
        # one decode step of a large continuous batch into FP8 caches, rows of the fused projection
        dict(name="append_step", kind="append", tokens=256, hq=64, hkv=8, d=128, bs=32, dtype="bf16",
             kv="fp8", rotary=128, interleaved=False, far=131072, rows="fused", k_scale=0.5, v_scale=0.25),
        # a prefill batch's chunks, some of the tokens padding without a slot
        dict(name="append_prompt", kind="append", tokens=16381, hq=32, hkv=8, d=128, bs=16, dtype="fp16",
             kv="16", rotary=128, interleaved=False, far=32768, rows="fused", k_scale=1.0, v_scale=1.0),
        # bounds: the blocks of a decode step's new tokens
        dict(name="bounds_step", kind="bounds", seqs=256, hq=64, hkv=8, d=128, bs=32, dtype="bf16",
             kv="16", lens="lognormal", lo=1, hi=16384, chunk=1, k_scale=1.0, v_scale=1.0),
        # the blocks of a prefill batch's chunks
        dict(name="bounds_prompt", kind="bounds", seqs=16, hq=32, hkv=8, d=128, bs=16, dtype="fp16",
             kv="fp8", lens="uniform", lo=1031, hi=4096, chunk=1031, k_scale=0.5, v_scale=1.0),
        # select: a step of four short sequences
        dict(name="select_tiny", kind="select", seqs=4, hq=4, hkv=4, d=64, bs=16, dtype="fp16",
             lens="uniform", lo=1, hi=200, chunk=1, keep=6, sink=1, recent=2),
        # drafted tokens scored against long contexts, each with blocks of its own
        dict(name="select_draft", kind="select", seqs=64, hq=32, hkv=8, d=128, bs=16, dtype="bf16",
             lens="uniform", lo=512, hi=4096, chunk=5, keep=32, sink=1, recent=2),
        # a step of a few very long sequences
        dict(name="select_long", kind="select", seqs=8, hq=32, hkv=8, d=128, bs=16, dtype="bf16",
             lens="long", lo=32768, hi=131072, chunk=1, keep=128, sink=4, recent=8),
        # sparse: 512 tokens for every sequence and KV head of an ordinary batch
        dict(name="sparse_batch", kind="sparse", seqs=64, hq=32, hkv=8, d=128, bs=16, dtype="fp16",
             kv="16", lens="uniform", lo=512, hi=4096, keep=32, k_scale=1.0, v_scale=1.0),
        # a large batch of mostly short sequences over FP8 caches: many have fewer blocks than may be kept
        dict(name="sparse_wide", kind="sparse", seqs=256, hq=64, hkv=8, d=128, bs=32, dtype="bf16",
             kv="fp8", lens="lognormal", lo=1, hi=16384, keep=32, k_scale=0.5, v_scale=0.7),
        # 2,048 tokens for every KV head of a few very long sequences
        dict(name="sparse_long", kind="sparse", seqs=8, hq=32, hkv=8, d=128, bs=16, dtype="bf16",
             kv="16", lens="long", lo=32768, hi=131072, keep=128, k_scale=1.0, v_scale=1.0),
        # a whole decode step of those: append, bounds, select, sparse
        dict(name="step_long", kind="step", seqs=8, hq=32, hkv=8, d=128, bs=16, dtype="bf16", kv="16",
             lens="long", lo=32768, hi=131072, chunk=1, keep=128, sink=4, recent=8, rotary=128,
             interleaved=False, far=131072, rows="fused", k_scale=1.0, v_scale=1.0),
    ]


def _between(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["append", "append", "bounds", "select", "select", "sparse", "sparse", "step"])
    d = rng.choice([64, 128])
    c = dict(kind=kind, d=d, bs=rng.choice([16, 32]), dtype=rng.choice(["fp16", "bf16"]),
             kv=rng.choice(["16", "fp8", "fp4"]), k_scale=rng.choice([1.0, 0.25, 0.7]),
             v_scale=rng.choice([1.0, 0.03125, 0.3]), hkv=rng.randint(1, 8))
    c["hq"] = c["hkv"] * rng.randint(1, 8)
    if kind in ("append", "step"):
        c.update(rotary=rng.choice([d, d, d // 2, 16, 48]), interleaved=rng.choice([False, True]),
                 rows=rng.choice(["packed", "fused"]), far=131072)
    if kind == "append":
        c.update(tokens=_between(rng, 1, 16381 * 48 // (c["hq"] + 2 * c["hkv"])))
        c["tokens"] = min(c["tokens"], 16381)
        return c
    if c["kv"] == "16":
        c.update(k_scale=1.0, v_scale=1.0)  # 16-bit caches have none
    hi = _between(rng, 1, 131072)
    seqs = _between(rng, 1, max(1, min(256, 360448 // hi)))
    c.update(seqs=seqs, lens="uniform", lo=rng.choice([0, 1, hi]), hi=hi)
    if kind == "bounds":
        c.update(chunk=rng.choice([1, _between(rng, 1, hi)]))
        # (no more keys than the largest listed case has)
        c["seqs"] = min(c["seqs"], max(1, 131072 // c["chunk"]))
        return c
    keep = _between(rng, 1, 2048 // c["bs"])
    c["seqs"] = min(c["seqs"], 262144 // (keep * c["bs"]))
    if kind in ("select", "step"):
        sink = rng.randint(0, min(4, keep))
        c.update(sink=sink, recent=rng.randint(0, min(8, keep - sink)))
        c.update(chunk=rng.choice([1, rng.randint(1, 8)]) if kind == "select" else 1)
        c["seqs"] = min(c["seqs"], max(1, 360448 // (hi * c["chunk"])))
    c.update(keep=keep)
    return c


# ------------------------------------------------------------------ the formats

def _e2m1(like):
    """The values of the sixteen codes."""
    m = torch.tensor(MAGNITUDES, dtype=like.dtype, device=like.device)
    return torch.cat([m, -m])


def _split(cache, bs, d):
    """The codes [.., bs, d / 2] and scales [.., bs, d / 16] of an FP4 cache, as views."""
    n = bs * (d // 2)
    return cache[..., :n].unflatten(-1, (bs, d // 2)), cache[..., n:].unflatten(-1, (bs, d // 16))


def _fp4(x, g):
    """(codes, scales) of rows x [..., d] in an FP4 cache of scale g."""
    x = x.float().unflatten(-1, (-1, 16))
    g = torch.full((), g, dtype=torch.float32, device=x.device)
    top = x.abs().amax(-1)
    s = (top / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    z = s.float() * g
    y = x * torch.ones_like(z).div(z).unsqueeze(-1)
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
            + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    code = code + 8 * torch.signbit(y).int()
    code = torch.where((z > 0).unsqueeze(-1), code, torch.zeros_like(code)).flatten(-2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), s.view(torch.uint8)


def _fp8(x, g):
    """E4M3 codes of x in an FP8 cache of scale g."""
    g = torch.full((), g, dtype=torch.float32, device=x.device)
    return (x.float() / g).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _stored(s, cache):
    """The values of (some blocks of) a cache without the cache's own scale, in 32 bits: [..., bs, d]."""
    if s["kv"] == "16":
        return cache.float()
    if s["kv"] == "fp8":
        return cache.view(torch.float8_e4m3fn).float()
    codes, scales = _split(cache, s["bs"], s["d"])
    e = _e2m1(torch.empty(0, device=cache.device))
    x = torch.stack([e[(codes & 15).int()], e[(codes >> 4).int()]], -1).flatten(-2)
    sc = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, 16)) * sc.unsqueeze(-1)).flatten(-2)


def _put(s, cache, at, x, g):
    """x, whole blocks [n, hkv, bs, d], into blocks `at` of a cache of scale g."""
    if s["kv"] == "16":
        cache[at] = x.to(cache.dtype)
    elif s["kv"] == "fp8":
        cache[at] = _fp8(x, g)
    else:
        codes, scales = _split(cache, s["bs"], s["d"])
        codes[at], scales[at] = _fp4(x, g)


def _empty(s, blocks):
    """A cache of zeros."""
    hkv, bs, d = s["hkv"], s["bs"], s["d"]
    size = (bs * d * 9 // 16,) if s["kv"] == "fp4" else (bs, d)
    return torch.zeros(blocks, hkv, *size, dtype=TYPES[s["dtype"]] if s["kv"] == "16" else torch.uint8, device="cuda")


def _pool(s, blocks, gen, g, mean, poison):
    """A cache with `blocks` blocks of N(mean, 1); `poison` [blocks]: the row of
    each from which on it holds NaN (bs: none)."""
    hkv, bs, d = s["hkv"], s["bs"], s["d"]
    cache = _empty(s, blocks)
    for at in torch.arange(blocks, device="cuda").split(4096):
        x = torch.randn(at.numel(), hkv, bs, d, generator=gen, device="cuda") + mean
        hide = torch.arange(bs, device="cuda") >= poison[at][:, None]
        _put(s, cache, at, torch.where(hide[:, None, :, None], math.nan, x), g)
    return cache


# ------------------------------------------------------------------- the inputs

def _lens(case, gen):
    """Context lengths.  A case has the same ones in another order for every
    seed, so that its caches and outputs keep their sizes."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    same = torch.Generator().manual_seed(1)
    if case["lens"] == "long":
        got = torch.full((n,), lo)
        got[-2], got[-1] = 2 * lo, hi
    elif case["lens"] == "lognormal":
        got = torch.randn(n, generator=same).add(math.log(1024)).exp().round().clamp(lo, hi).long()
    else:
        got = torch.randint(lo, hi + 1, (n,), generator=same)
    return got[torch.randperm(n, generator=gen)]


def _rows(s, n, gen):
    """Queries, keys and values of n new tokens: tensors of their own, or views
    of the rows of a fused projection."""
    hq, hkv, d, t = s["hq"], s["hkv"], s["d"], TYPES[s["dtype"]]
    both = torch.randn(n, hq + 2 * hkv, d, generator=gen, device="cuda").to(t)
    parts = both[:, :hq], both[:, hq:hq + hkv], both[:, hq + hkv:]
    s["query"], s["key"], s["value"] = parts if s["rows"] == "fused" else [x.contiguous() for x in parts]
    s["query_out"] = torch.zeros(n, hq, d, dtype=t, device="cuda")
    # a model's own table of angles
    half = s["rotary"] // 2
    freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = torch.arange(s["far"], device="cuda", dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    s = dict(case)
    s.setdefault("kv", "16")
    if s["kind"] == "append":
        n = s["tokens"]
        blocks = -(-n // bs) + 3
        order = torch.randperm(blocks, generator=host)  # consecutive tokens, in blocks scattered over the pool
        j = torch.arange(n)
        slots = order[j // bs] * bs + j % bs
        if n > 16:
            slots[torch.randperm(n, generator=host)[: n // 16]] = -1  # padding tokens
        run = max(1, n // 16)  # tokens in a row of one sequence (a step's: one)
        first = torch.randint(0, max(1, s["far"] - run), (n // run + 1,), generator=host)
        s["slots"] = slots.cuda()
        s["positions"] = (first[j // run] + j % run).clamp(max=s["far"] - 1).cuda()
        _rows(s, n, gen)
        s["k_cache"], s["v_cache"] = _empty(s, blocks), _empty(s, blocks)
        if s["kv"] == "fp4":
            s["out_k"] = torch.zeros(n, hkv, d, dtype=TYPES[s["dtype"]], device="cuda")
            s["out_v"] = torch.zeros_like(s["out_k"])
        return s
    lens = _lens(case, host)
    per = (lens + bs - 1) // bs
    used = int(per.sum())
    blocks = used + used // 10 + 1
    order = torch.randperm(blocks, generator=host)[:used]
    width = max(1, int(per.max()))
    have = torch.arange(width) < per[:, None]
    table = torch.full((lens.numel(), width), -1)
    table[have] = order  # row by row: every sequence its own blocks
    tail = torch.full((blocks,), 0)
    tail[order] = bs
    some = lens > 0
    tail[table[some, per[some] - 1]] = (lens[some] - 1) % bs + 1
    s["tables"], s["ctx"] = table.int().cuda(), lens.int().cuda()
    s["longest"] = int(lens.max())
    mean = 2.0 * torch.randn(1, hkv, 1, d, generator=gen, device="cuda")  # keys have channels of their own
    poison = tail.cuda() if s["kind"] != "step" else torch.full((blocks,), bs, device="cuda")
    s["k_cache"] = _pool(s, blocks, gen, s.get("k_scale", 1.0), mean, poison)
    if s["kind"] in ("sparse", "step"):
        s["v_cache"] = _pool(s, blocks, gen, s["v_scale"], 0.0, poison)
        s["scale"] = 1.0 / math.sqrt(d)
    if s["kind"] != "sparse":
        s["bounds"] = torch.zeros(blocks, hkv, 2, d, dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros(blocks, hkv, dtype=torch.float32, device="cuda")
    if s["kind"] in ("select", "step"):
        for at in torch.arange(blocks, device="cuda").split(4096):  # a serving loop has kept them up
            full = torch.where(tail.cuda()[at] > 0, tail.cuda()[at], bs)
            s["bounds"][at], s["scales"][at] = _extremes(_stored(s, s["k_cache"][at]), full)
    if s["kind"] == "select":
        del s["k_cache"]  # the call looks at the bounds alone
    rows = lens.numel()
    if s["kind"] in ("bounds", "select"):
        q = lens.clamp(max=s["chunk"])
        start = torch.zeros(q.numel() + 1, dtype=torch.long)
        start[1:] = q.cumsum(0)
        s["longest_q"] = max(1, int(q.max()))
        if s["chunk"] > 1:
            s["start"], rows = start.int().cuda(), int(start[-1])
    if s["kind"] in ("select", "sparse"):
        s["query"] = torch.randn(rows, hq, d, generator=gen, device="cuda").to(TYPES[s["dtype"]])
        if s["kind"] == "sparse":
            s["out"] = torch.zeros_like(s["query"])
    if s["kind"] == "step":
        _rows(s, rows, gen)
        s["positions"] = (lens - 1).clamp(min=0).cuda()
        at = table[torch.arange(rows), (per - 1).clamp(min=0)]
        s["slots"] = torch.where(some, at * bs + (lens - 1) % bs, -1).cuda()
        s["out"] = torch.zeros_like(s["query_out"])
    if s["kind"] in ("select", "step"):
        s["picked"] = torch.zeros(rows, hkv, s["keep"], dtype=torch.int32, device="cuda")
        s["picked_lens"] = torch.zeros(rows, hkv, dtype=torch.int32, device="cuda")
    if s["kind"] == "sparse":
        # some blocks of each sequence for each head, the last one always, in order
        r = torch.rand(rows, hkv, width, generator=gen, device="cuda")
        n = per.cuda()[:, None, None]
        j = torch.arange(width, device="cuda")
        r = torch.where(j < n, r, 2.0)
        r = torch.where(j == n - 1, -1.0, r)
        keep = min(s["keep"], width)
        got = r.argsort(-1)[..., :keep].sort(-1).values
        ok = got < n
        ids = s["tables"].long()[torch.arange(rows, device="cuda")[:, None, None], got]
        s["picked"] = torch.full((rows, hkv, s["keep"]), -1, dtype=torch.int32, device="cuda")
        s["picked"][..., :keep] = torch.where(ok, ids, -1).int()
        last = (s["ctx"][:, None] - 1) % bs + 1
        s["picked_lens"] = torch.where(s["ctx"][:, None] > 0, (ok.sum(-1) - 1) * bs + last, 0).int()
    return s


# ---------------------------------------------------------------- the operators

def _pow2(e):
    """2^e of whole numbers of -126..127, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _exponent(a, most):
    """The smallest e >= -126 with a <= most 2^e, for finite a > 0 and most = 2^n - 1."""
    m, x = torch.frexp(a)  # a = m 2^x, 0.5 <= m < 1
    n = most.bit_length()
    return (x - n + (m > most / 2 ** n).int()).clamp(min=-126)


def _rotate(s, x):
    """Rows [T, heads, d] at their positions, rounded to their type."""
    r, half = s["rotary"], s["rotary"] // 2
    cs = s["cos_sin"][s["positions"].clamp(0, s["far"] - 1)][:, None]
    cos, sin = cs[..., :half], cs[..., half:]
    v = x[..., :r].float()
    if s["interleaved"]:
        a, b = v[..., 0::2], v[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = v[..., :half], v[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned.to(x.dtype), x[..., r:]], -1)


def _append(s):
    keep = s["slots"] >= 0  # a padding token leaves what is at its place
    at, row = s["slots"][keep] // s["bs"], s["slots"][keep] % s["bs"]
    s["query_out"][keep] = _rotate(s, s["query"])[keep]
    for cache, x, g in ((s["k_cache"], _rotate(s, s["key"]), s["k_scale"]),
                        (s["v_cache"], s["value"], s["v_scale"])):
        if s["kv"] == "16":
            cache[at, :, row] = x[keep]
        elif s["kv"] == "fp8":
            cache[at, :, row] = _fp8(x[keep], g)
        else:
            codes, scales = _split(cache, s["bs"], s["d"])
            codes[at, :, row], scales[at, :, row] = _fp4(x[keep], g)


def _read_back(s, cache, out, g):
    """An FP4 cache's rows at the slots, in the rows' type."""
    codes, scales = _split(cache, s["bs"], s["d"])
    at = s["slots"].clamp(min=0)
    at, row = at // s["bs"], at % s["bs"]
    sc = scales[at, :, row].contiguous().view(torch.float8_e4m3fn).float() * g
    c = codes[at, :, row]
    e = _e2m1(sc)
    x = torch.stack([e[(c & 15).int()], e[(c >> 4).int()]], -1).flatten(-2)
    x = (x.unflatten(-1, (-1, 16)) * sc.unsqueeze(-1)).flatten(-2).to(out.dtype)
    return torch.where((s["slots"] >= 0)[:, None, None], x, out)


def _appended(s):
    """What append gives: of 8-bit caches the values of the codes (as that type), of 4-bit ones the rows."""
    if s["kv"] == "fp4":
        return [s["query_out"], s["out_k"], s["out_v"]]
    caches = [s["k_cache"], s["v_cache"]]
    return [s["query_out"]] + [c.view(torch.float8_e4m3fn) if s["kv"] == "fp8" else c for c in caches]


def _extremes(x, full):
    """(codes [n, hkv, 2, d], scales [n, hkv]) of blocks x [n, hkv, bs, d] whose first `full` rows count."""
    use = (torch.arange(x.shape[2], device=x.device) < full[:, None])[:, None, :, None]
    hi, lo = torch.where(use, x, -math.inf).amax(2), torch.where(use, x, math.inf).amin(2)
    a = torch.where(use, x.abs(), 0.0).amax((2, 3))  # NaN where one of them is
    fine = a < math.inf
    e = _exponent(torch.where(fine & (a > 0), a, 1.0), 127)
    up = _pow2(-e)[..., None]
    some = (fine & (a > 0))[..., None]
    codes = torch.stack([torch.where(some, (hi * up).ceil(), 0.0),
                         torch.where(some, (lo * up).floor(), 0.0)], 2).to(torch.int8)
    return codes, torch.where(fine, torch.where(a > 0, _pow2(e), 0.0), math.inf)


def _bounds(s):
    bs, ctx = s["bs"], s["ctx"].long()
    new = ctx.clamp(max=s["chunk"]) if s["kind"] == "bounds" else ctx.clamp(max=1)
    j = torch.arange(s["tables"].shape[1], device="cuda")
    touched = (j >= (ctx - new)[:, None] // bs) & (j * bs < ctx[:, None]) & (new > 0)[:, None]
    seq, j = touched.nonzero(as_tuple=True)
    at = s["tables"][seq, j].long()
    full = (ctx[seq] - j * bs).clamp(max=bs)
    s["bounds"][at], s["scales"][at] = _extremes(_stored(s, s["k_cache"][at]), full)


def _of_rows(s):
    """The sequence of each row, and the tokens it sees."""
    ctx = s["ctx"].long()
    if "start" not in s:
        return torch.arange(ctx.numel(), device="cuda"), ctx
    start = s["start"].long()
    row = torch.arange(s["query"].shape[0], device="cuda")
    seq = torch.searchsorted(start[1:], row, right=True)
    return seq, ctx[seq] - (start[seq + 1] - 1 - row)


def _select(s, query):
    """(tables, lengths)"""
    bs, keep = s["bs"], s["keep"]
    seq, seen = _of_rows(s)
    n = ((seen + bs - 1) // bs)[:, None, None]
    q = query.float().unflatten(1, (s["hkv"], -1))  # [rows, kv heads, group, d]
    a = q.abs().amax((2, 3))
    ok = (a < math.inf) & (a > 0)
    e = _exponent(torch.where(ok, a, 1.0), 4095)
    c = torch.where(ok[..., None, None], (q * _pow2(-e)[..., None, None]).round(), 0.0).double()
    w = torch.stack([c.clamp(min=0).sum(2), c.clamp(max=0).sum(2)], 2).flatten(2)  # whole numbers in 64 bits
    at = s["tables"][seq].long().clamp(min=0)  # [rows, blocks]
    b = s["bounds"][at].transpose(1, 2).flatten(3).double()
    total = (b @ w.unsqueeze(-1)).squeeze(-1).float()
    scale = s["scales"][at].transpose(1, 2)
    score = torch.where(scale == math.inf, math.inf, total * torch.where(scale == math.inf, 1.0, scale))
    score = score.double().clamp(-1e300, 1e300)
    j = torch.arange(at.shape[1], device="cuda")
    score = torch.where((j < s["sink"]) | (j >= n - s["recent"]), math.inf, score)
    score = torch.where(j < n, score, -math.inf)
    got = score.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    got = torch.where(got < n, got, at.shape[1]).sort(-1).values
    real = got < n
    ids = torch.where(real, at.unsqueeze(1).expand(-1, s["hkv"], -1).gather(
        2, got.clamp(max=at.shape[1] - 1)), -1).int()
    tables = torch.full_like(s["picked"], -1)
    tables[..., :ids.shape[-1]] = ids
    short = (real & (got == n - 1)).any(-1) * (n[..., 0] * bs - seen[:, None])
    return tables, (real.sum(-1) * bs - short).int()


def _attend(s, query, tables, lens):
    """Softmax attention of every row over the blocks of its tables."""
    q = query.float().unflatten(1, (s["hkv"], -1))  # [rows, kv heads, group, d]
    at = tables.clamp(min=0).long()
    head = torch.arange(s["hkv"], device="cuda")[:, None]
    k = (_stored(s, s["k_cache"][at, head]) * s["k_scale"]).flatten(2, 3)  # [rows, kv heads, tokens, d]
    v = (_stored(s, s["v_cache"][at, head]) * s["v_scale"]).flatten(2, 3)
    seen = torch.arange(k.shape[2], device="cuda") < lens[..., None]
    z = torch.where(seen[:, :, None], (q @ k.transpose(-1, -2)) * s["scale"], -math.inf)
    top = z.amax(-1, keepdim=True)
    e = (z - torch.where(top == -math.inf, 0.0, top)).exp()
    total = e.sum(-1, keepdim=True)
    o = (e / torch.where(total == 0, 1.0, total)) @ torch.where(seen[..., None], v, 0.0)
    return o.flatten(1, 2).to(query.dtype)


def run(state):
    s = state
    kind = s["kind"]
    if own:
        return _run_own(s)
    if kind == "append":
        _append(s)
        if s["kv"] == "fp4":
            s["out_k"] = _read_back(s, s["k_cache"], s["out_k"], s["k_scale"])
            s["out_v"] = _read_back(s, s["v_cache"], s["out_v"], s["v_scale"])
        return _appended(s)
    if kind == "bounds":
        _bounds(s)
        return [s["bounds"], s["scales"]]
    if kind == "select":
        return _select(s, s["query"])
    if kind == "sparse":
        return _attend(s, s["query"], s["picked"], s["picked_lens"])
    _append(s)
    _bounds(s)
    tables, lens = _select(s, s["query_out"])
    out = _attend(s, s["query_out"], tables, lens)
    return {"tables": tables, "lens": lens, "out": out, "query": s["query_out"],
            "bounds": s["bounds"], "scales": s["scales"],
            **({} if s["kv"] == "fp4" else dict(zip("kv", _appended(s)[1:])))}


def _run_own(s):
    import pagedattention_kv_cache_attention_gb300 as pa
    kind, end = s["kind"], {"16": "", "fp8": "_fp8", "fp4": "_fp4"}[s["kv"]]
    pair = () if s["kv"] == "16" else (s.get("k_scale", 1.0), s.get("v_scale", 1.0))
    if kind in ("append", "step"):
        getattr(pa, "pa_rope_and_cache" + end)(
            s["query_out"], s["query"], s["key"], s["value"], s["k_cache"], s["v_cache"], s["slots"],
            s["positions"], s["cos_sin"], *pair, interleaved=s["interleaved"])
        if kind == "append":
            if s["kv"] == "fp4":
                pa.pa_gather_cache_fp4(s["out_k"], s["out_v"], s["k_cache"], s["v_cache"], s["slots"], *pair)
            return _appended(s)
    if kind in ("bounds", "step"):
        getattr(pa, "pa_update_key_bounds" + end)(s["bounds"], s["scales"], s["k_cache"], s["tables"],
                                                  s["ctx"], s.get("start"), s.get("longest_q", 1))
        if kind == "bounds":
            return [s["bounds"], s["scales"]]
    query = s["query_out"] if kind == "step" else s["query"]
    if kind in ("select", "step"):
        pa.pa_select_blocks(s["picked"], s["picked_lens"], query, s["bounds"], s["scales"], s["tables"],
                            s["ctx"], s["bs"], s["longest"], s["sink"], s["recent"], s.get("start"),
                            s.get("longest_q", 1))
        if kind == "select":
            return s["picked"], s["picked_lens"]
    getattr(pa, "pa_decode_sparse" + end)(s["out"], query, s["k_cache"], s["v_cache"], s["picked"],
                                          s["picked_lens"], s["scale"], *pair)
    if kind == "sparse":
        return s["out"]
    return {"tables": s["picked"], "lens": s["picked_lens"], "out": s["out"], "query": s["query_out"],
            "bounds": s["bounds"], "scales": s["scales"],
            **({} if s["kv"] == "fp4" else dict(zip("kv", _appended(s)[1:])))}


# ---------------------------------------------------- the definition in 64 bits

def _to32(x):
    return x.float().double()


def _turned(s, x):
    """Rotated rows in 64 bits, with the definition's roundings: pair by pair, from exact products."""
    half = s["rotary"] // 2
    cs = s["cos_sin"].double()[s["positions"].clamp(0, s["far"] - 1)]
    out = x.double()
    i = torch.arange(half, device="cuda")
    p, q = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
    a, b, cos, sin = out[..., p], out[..., q], cs[:, None, :half], cs[:, None, half:]
    turned = out.clone()
    turned[..., p] = _to32(_to32(a * cos) - _to32(b * sin))
    turned[..., q] = _to32(_to32(b * cos) + _to32(a * sin))
    return turned


def _e4m3_of(x):
    """The nearest E4M3 value (ties to even, at most 448) of values in 64 bits, by a search over all of them."""
    k = torch.arange(127, device=x.device)
    grid = torch.where(k < 8, k * 2.0 ** -9, (1 + (k & 7) / 8) * torch.exp2(((k >> 3) - 7).double()))
    mid = (grid[1:] + grid[:-1]) / 2
    a = x.abs().clamp(max=448.0)
    at = torch.searchsorted(mid, a)
    tie = (at < 126) & (mid[at.clamp(max=125)] == a) & (at % 2 == 1)
    return grid[at + tie.long()] * torch.sign(x)


def _e4m3_bits(raw):
    raw = raw.long()
    expo, frac = (raw >> 3) & 15, (raw & 7).double()
    v = torch.where(expo == 0, frac * 2.0 ** -9, (1 + frac / 8) * torch.exp2((expo - 7).double()))
    v = torch.where((raw & 127) == 127, math.nan, v)
    return torch.where(raw >= 128, -v, v)


def _held(s, cache):
    """The values of blocks of a cache in 64 bits, from the bits, without the cache's own scale."""
    if s["kv"] == "16":
        return cache.double()
    if s["kv"] == "fp8":
        return _e4m3_bits(cache)
    bs, d = s["bs"], s["d"]
    n = bs * d // 2
    raw = cache[..., :n].reshape(*cache.shape[:-1], bs, d // 2).long()
    nib = torch.stack([raw & 15, raw >> 4], -1).flatten(-2)
    e, m = (nib >> 1) & 3, (nib & 1).double()
    x = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).double()))
    sc = _e4m3_bits(cache[..., n:].reshape(*cache.shape[:-1], bs, d // 16))
    return torch.where(nib >= 8, -x, x) * torch.repeat_interleave(sc, 16, -1)


def _fp4_held(x, g):
    """What rows read back as from an FP4 cache, in 64 bits."""
    g = torch.tensor(g, dtype=torch.float32).double().item()
    b = x.double().unflatten(-1, (-1, 16))
    six = torch.tensor(6.0 * g, dtype=torch.float64).float().double().item()
    sc = _e4m3_of(_to32(b.abs().amax(-1) / six))
    inv = _to32(1.0 / _to32(sc * g))
    y = _to32(b * inv.unsqueeze(-1))
    mags = torch.tensor(MAGNITUDES, dtype=torch.float64, device=b.device)
    cut = (mags[1:] + mags[:-1]) / 2
    i = torch.searchsorted(cut, y.abs())
    tie = (i < 7) & (cut[i.clamp(max=6)] == y.abs()) & (i % 2 == 1)
    v = torch.where((sc > 0).unsqueeze(-1), mags[i + tie.long()] * torch.sign(y), 0.0)
    return (v * sc.unsqueeze(-1) * g).flatten(-2)


def _caches_after(s):
    """What append leaves: queries and both caches (or the rows read back from FP4 ones), in 64 bits."""
    t = TYPES[s["dtype"]]
    keep = s["slots"] >= 0
    at, row = s["slots"][keep] // s["bs"], s["slots"][keep] % s["bs"]
    got = [torch.where(keep[:, None, None], _turned(s, s["query"]).to(t).double(), s["query_out"].double())]
    for cache, x, g in ((s["k_cache"], _turned(s, s["key"]).to(t).double(), s["k_scale"]),
                        (s["v_cache"], s["value"].double(), s["v_scale"])):
        if s["kv"] == "fp4":
            got.append(torch.where(keep[:, None, None], _fp4_held(x, g), 0.0))
            continue
        held = _held(s, cache)
        g = torch.tensor(g, dtype=torch.float32).double().item()
        held[at, :, row] = x[keep] if s["kv"] == "16" else _e4m3_of(_to32(x[keep] / g))
        got.append(held)
    return got


def _scales_after(s, keys):
    """The bounds and scales after the call, keys being the K cache's values in 64 bits."""
    bounds, scales = s["bounds"].cpu().numpy().copy(), s["scales"].double().cpu().numpy()
    for i, n in enumerate(s["ctx"].tolist()):
        new = min(n, s["chunk"])
        for j in range((n - new) // s["bs"], -(-n // s["bs"])) if new else ():
            at = int(s["tables"][i, j])
            x = keys[at][:, : n - j * s["bs"]].cpu().numpy()
            for h in range(s["hkv"]):
                a = np.abs(x[h]).max()
                if not np.isfinite(a):
                    bounds[at, h], scales[at, h] = 0, math.inf
                    continue
                e = max(-126, math.ceil(math.log2(a / 127.0))) if a else 0
                e += a > 127.0 * 2.0 ** e
                e -= a <= 127.0 * 2.0 ** (e - 1) and e > -126
                scales[at, h] = 2.0 ** e if a else 0.0
                bounds[at, h] = np.stack([np.ceil(x[h].max(0) / 2.0 ** e), np.floor(x[h].min(0) / 2.0 ** e)])
    return bounds, scales


def _chosen(s, query, bounds, scales):
    """Tables and lengths, row by row in numpy."""
    bs, keep = s["bs"], s["keep"]
    seq, seen = (x.cpu().numpy() for x in _of_rows(s))
    q = query.double().cpu().numpy().reshape(len(seq), s["hkv"], -1, s["d"])
    table = s["tables"].cpu().numpy()
    ids, lens = np.full((len(seq), s["hkv"], keep), -1), np.zeros((len(seq), s["hkv"]), np.int64)
    for r, (i, tokens) in enumerate(zip(seq, seen)):
        n = -(-int(tokens) // bs)
        at = table[i, :n]
        for h in range(s["hkv"] if n else 0):
            a = np.abs(q[r, h]).max()
            e = 0
            while a > 4095.0 * 2.0 ** e:
                e += 1
            while a and e > -126 and a <= 4095.0 * 2.0 ** (e - 1):
                e -= 1
            c = np.rint(q[r, h] / 2.0 ** e).astype(np.int64)
            b = bounds[at, h].astype(np.int64)
            total = b[:, 0] @ np.maximum(c, 0).sum(0) + b[:, 1] @ np.minimum(c, 0).sum(0)
            score = (total.astype(np.float32) * scales[at, h].astype(np.float32)).astype(np.float64)
            score[: s["sink"]] = math.inf
            score[n - min(n, s["recent"]):] = math.inf
            got = np.sort(np.lexsort((np.arange(n), -score))[:keep])
            ids[r, h, : len(got)] = at[got]
            lens[r, h] = len(got) * bs - (n * bs - tokens if got[-1] == n - 1 else 0)
    return torch.from_numpy(ids).cuda(), torch.from_numpy(lens).cuda()


def _attended(s, query, tables, lens, keys=None, values=None):
    """Attention in 64 bits, a row at a time."""
    group = s["hq"] // s["hkv"]
    ks, vs = (torch.tensor(s[g], dtype=torch.float32).double().item() for g in ("k_scale", "v_scale"))
    head = torch.arange(s["hkv"], device="cuda")[:, None]
    out = torch.zeros(query.shape, dtype=torch.float64, device="cuda")
    for r in range(query.shape[0]):
        at = tables[r].long().clamp(min=0)
        k, v = ((_held(s, cache[at, head]) if held is None else held[at, head]).flatten(1, 2)
                for cache, held in ((s["k_cache"], keys), (s["v_cache"], values)))
        hide = torch.arange(k.shape[1], device="cuda") >= lens[r][:, None]
        z = query[r].double().unflatten(0, (-1, group)) @ (k * ks).transpose(1, 2) * s["scale"]
        p = torch.softmax(z.masked_fill(hide[:, None], -math.inf), -1)
        p = torch.where(lens[r][:, None, None] > 0, p, 0.0)
        out[r] = (p @ (v * vs).masked_fill(hide[..., None], 0.0)).flatten(0, 1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "append":
        return _caches_after(s)
    if s["kind"] == "bounds":
        bounds, scales = _scales_after(s, _held(s, s["k_cache"]))
        return [torch.from_numpy(bounds), torch.from_numpy(scales)]
    if s["kind"] == "select":
        return _chosen(s, s["query"], s["bounds"].cpu().numpy(), s["scales"].cpu().numpy())
    if s["kind"] == "sparse":
        return _attended(s, s["query"], s["picked"], s["picked_lens"])
    if s["kv"] == "fp4":
        return None  # the cache's own values are what append's cases look at
    q, keys, values = _caches_after(s)
    s["chunk"] = 1
    bounds, scales = _scales_after(s, keys)
    tables, lens = _chosen(s, q, bounds, scales)
    return {"tables": tables, "lens": lens, "out": _attended(s, q, tables, lens, keys, values), "query": q,
            "bounds": torch.from_numpy(bounds), "scales": torch.from_numpy(scales), "k": keys, "v": values}


# -------------------------------------------------------------------- the work

def _bytes_of(case):
    """Bytes of a cached element."""
    return {"16": 2.0, "fp8": 1.0, "fp4": 9.0 / 16}[case.get("kv", "16")]


def work(case):
    d, hq, hkv, bs, kind = case["d"], case["hq"], case["hkv"], case["bs"], case["kind"]
    moved = flops = 0.0
    if kind != "append":
        lens = _lens(case, torch.Generator()).double()
        tokens = float(lens.clamp(max=case.get("chunk", 1)).sum())
    else:
        tokens = case["tokens"] * (15 / 16 if case["tokens"] > 16 else 1)
    if kind in ("append", "step"):
        # rows in, queries and cached rows out, a row of the table, slot and position
        moved += tokens * ((2 * hq + 2 * hkv) * d * 2 + 2 * hkv * d * _bytes_of(case) + case["rotary"] * 4 + 16)
        flops += tokens * (hq + hkv) * case["rotary"] * 3
        if case["kv"] == "fp4" and kind == "append":
            moved += tokens * 2 * hkv * d * 2  # read back as 16-bit rows
    if kind in ("bounds", "step"):
        new = lens.clamp(max=case["chunk"])
        first = torch.floor((lens - new) / bs)
        keys = float((lens - first * bs)[new > 0].sum())
        blocks = float((torch.ceil(lens / bs) - first)[new > 0].sum())
        moved += hkv * (keys * d * _bytes_of(case) + blocks * (2 * d + 4)) + blocks * 4
        flops += keys * hkv * d * 3
    if kind in ("select", "step"):
        blocks = torch.ceil(lens / bs)
        kept = float((blocks.clamp(max=case["keep"]) * lens.clamp(max=case["chunk"])).sum())
        moved += float(blocks.sum()) * (hkv * (2 * d + 4) + 4) + tokens * (hq * d * 2 + hkv * 4) + kept * hkv * 4
        flops += float((blocks * lens.clamp(max=case["chunk"])).sum()) * hkv * 4 * d
    if kind in ("sparse", "step"):
        blocks = torch.ceil(lens / bs).clamp(max=case["keep"])
        read = float(torch.minimum(blocks * bs, lens).sum())
        moved += read * hkv * 2 * d * _bytes_of(case) + float(blocks.sum()) * hkv * 4 + 2 * lens.numel() * hq * d * 2
        flops += 4.0 * read * hq * d
    return {"bytes": moved, "flops": flops}
