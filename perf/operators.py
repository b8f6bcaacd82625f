"""Cases of the paged 8-bit cache: append, attention, attention weights, eviction.

The cache holds K and V in 8 bits (int8 or e4m3), in pages of 64 tokens, with one
float32 scale for each page and head; a block table gives each sequence its pages.

`own` false: every operator in its plain form, elementary torch operations on
dense tensors gathered from the pages. `own` true: the calls a user makes.
"""
import math

import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}

# Bounds of the drawn cases, the largest listed ones' cost: score matrix entries
# of a pass, and elements of K that a pass reads or writes.
MOST_SCORES = 2 * 16 * 4096 * 10521
MOST_ELEMENTS = 32 * 8 * 10521 * 128


def _case(name, op, **over):
    c = {"name": name, "op": op, "batch": 1, "q_heads": 16, "kv_heads": 16, "head_dim": 128, "fmt": "int8",
         "dtype": "bf16", "n": 1, "tokens": 680, "ragged": False, "causal": False, "prefix": 0, "docs": 0,
         "softcap": 0.0, "slopes": False, "evicted": False, "keep": 0, "sinks": 0, "recent": 0}
    c.update(over)
    return c


def listed():
    return [
        # one new token of each of 64 sequences, each at its own place in a page: the append of a decoding step
        _case("append_token", "append", batch=64, kv_heads=8, tokens=10521, ragged=True),
        # a chunk of three video frames (4680 tokens) behind a ragged past: the append of a next-frame step
        _case("append_chunk", "append", batch=4, kv_heads=12, fmt="e4m3", n=4680, tokens=18720, ragged=True),
        # one sequence, one token, a short image sequence: the smallest call, latency alone
        _case("attention_token", "attention", head_dim=64, tokens=680),
        # a batch of ragged sequences with shared key heads, one token each: ordinary serving
        _case("attention_batch", "attention", batch=32, q_heads=32, kv_heads=8, tokens=10521, ragged=True),
        # one very long sequence with capped scores and a distance bias: few rows, a long axis
        _case("attention_long", "attention", q_heads=32, kv_heads=4, fmt="e4m3", dtype="fp16", tokens=131071,
              softcap=50.0, slopes=True),
        # six drafted tokens to verify at once, over caches that were evicted from before (positions with gaps)
        _case("attention_draft", "attention", batch=8, q_heads=24, kv_heads=12, fmt="e4m3", n=6, tokens=9360,
              ragged=True, causal=True, slopes=True, evicted=True),
        # the last scale of a next-scale image model: 4096 queries that all see 10521 tokens
        _case("attention_block", "attention", batch=2, n=4096, tokens=10521),
        # a prompt chunk behind a past, documents packed into one sequence, capped scores, shared key heads, odd sizes
        _case("attention_prompt", "attention", q_heads=32, kv_heads=8, dtype="fp16", n=4097, tokens=8191, causal=True,
              docs=2048, softcap=30.0),
        # the weights that one decoding step adds to a ragged batch of caches
        _case("weights_token", "weights", batch=32, q_heads=32, kv_heads=8, tokens=10521, ragged=True),
        # the weights that the queries of one video frame give to a window of twelve frames, a prefix seen by all
        _case("weights_frame", "weights", batch=2, q_heads=12, kv_heads=12, fmt="e4m3", n=1560, tokens=18720,
              causal=True, prefix=77),
        # a handful of short sequences down to a small budget
        _case("evict_short", "evict", batch=4, kv_heads=8, head_dim=64, tokens=1021, ragged=True, keep=384, sinks=4,
              recent=64),
        # a video window of twelve frames down to six, the last frame always kept
        _case("evict_window", "evict", batch=8, kv_heads=12, fmt="e4m3", tokens=18720, keep=9360, sinks=16,
              recent=1560),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "weights", "evict"])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 12, 16])
    group = rng.choice([1, 1, 2, 3, 4, 8]) if op in ("attention", "weights") else 1
    c = _case("", op, kv_heads=kv_heads, q_heads=kv_heads * group, head_dim=rng.choice([64, 128]),
              fmt=rng.choice(["int8", "e4m3"]), dtype=rng.choice(["bf16", "bf16", "fp16"]), ragged=rng.random() < 0.7)
    del c["name"]
    c["tokens"] = _spread(rng, 30, 40000)
    c["batch"] = _spread(rng, 1, 48)
    most = MOST_ELEMENTS // (kv_heads * c["head_dim"])
    if op == "append":
        c["dtype"] = rng.choice(["bf16", "fp16", "f32"])
        c["n"] = rng.choice([1, rng.randint(2, 70), _spread(rng, 64, 8000)])
        c["tokens"] = max(c["tokens"], c["n"])
        c["batch"] = max(1, min(c["batch"], most // max(c["n"], 1) // 8, most // c["tokens"]))
        return c
    c["batch"] = max(1, min(c["batch"], most // c["tokens"]))
    if op == "evict":
        c["keep"] = max(1, int(c["tokens"] * rng.uniform(0.1, 1.05)))
        c["sinks"] = rng.choice([0, min(4, c["keep"])])
        c["recent"] = rng.randint(0, (c["keep"] - c["sinks"]) // 2)
        return c
    c["n"] = rng.choice([1, 1, rng.randint(2, 17), _spread(rng, 16, 4200)])
    c["n"] = min(c["n"], c["tokens"])
    c["batch"] = max(1, min(c["batch"], MOST_SCORES // (c["q_heads"] * c["n"] * c["tokens"])))
    c["n"] = max(1, min(c["n"], MOST_SCORES // (c["batch"] * c["q_heads"] * c["tokens"])))
    c["causal"] = rng.random() < 0.6
    c["softcap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
    c["slopes"] = rng.random() < 0.3
    c["evicted"] = rng.random() < 0.3
    c["prefix"] = rng.choice([0, 0, rng.randint(1, c["tokens"])]) if c["causal"] else 0
    c["docs"] = rng.choice([0, 0, max(8, c["tokens"] // 4)])
    return c


def _lens(c, g):
    """Cached tokens of each sequence, the call's own among them."""
    low = max(c["n"], c["tokens"] // 4) if c["ragged"] else c["tokens"]
    lens = torch.randint(low, c["tokens"] + 1, (c["batch"],), generator=g, device="cuda", dtype=torch.int32)
    lens[0] = c["tokens"]
    return lens


def _codes(shape, fmt, g):
    """Codes of a cache in use: a few channels of large values, the others small, every place filled."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
    wide = torch.ones(shape[-1], device="cuda", dtype=torch.float16)
    wide[torch.randperm(shape[-1], generator=g, device="cuda")[:max(1, shape[-1] // 16)]] = 6.0
    x.mul_(wide)
    if fmt == "int8":
        return x.mul_(9.0).round_().clamp_(-127, 127).to(torch.int8)
    return x.mul_(30.0).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _scales(shape, fmt, g):
    s = torch.exp(0.4 * torch.randn(shape, generator=g, device="cuda")) * (0.06 if fmt == "int8" else 0.015)
    return s if fmt == "int8" else torch.exp2(torch.floor(torch.log2(s)))


def _pools(c, g, lens, extra=0):
    """The cache, its block table, and what older sequences left behind in it: places that no
    sequence holds have any code, NaN among them, and pages of none have NaN for a scale."""
    B, H, D = c["batch"], c["kv_heads"], c["head_dim"]
    per = -(-c["tokens"] // PAGE)
    pages = B * per + 3
    s = {"k": _codes((pages, H, PAGE, D), c["fmt"], g), "v": _codes((pages, H, PAGE, D), c["fmt"], g),
         "k_scale": _scales((pages, H), c["fmt"], g), "v_scale": _scales((pages, H), c["fmt"], g)}
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = order[:B * per].reshape(B, per).contiguous()
    spare = order[B * per:].long()
    if c["fmt"] == "e4m3":
        for name in ("k", "v"):
            raw = s[name].view(torch.uint8)
            raw[spare] = 0x7F
            last = (lens.long() - 1) // PAGE
            page = table.long()[torch.arange(B, device="cuda"), last]
            behind = torch.arange(PAGE, device="cuda")[None, :] > ((lens.long() - 1) % PAGE)[:, None]
            raw[page] = torch.where(behind[:, None, :, None], torch.full_like(raw[page], 0x7F), raw[page])
    s["k_scale"][spare] = float("nan")
    s["v_scale"][spare] = float("nan")
    used = torch.arange(per, device="cuda")[None, :] * PAGE < lens[:, None]
    s["table"] = torch.where(used, table, torch.full_like(table, -1))
    if extra:
        s["table"] = table
    return s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, H, Hq, D, n = c["batch"], c["kv_heads"], c["q_heads"], c["head_dim"], c["n"]
    dtype = DTYPES[c["dtype"]]
    lens = _lens(c, g)
    s = _pools(c, g, lens, extra=c["op"] == "append")
    s.update(case=c, lens=lens, pos=None, weight=None)
    per = s["table"].shape[1]
    pages = s["k"].shape[0]
    if c["op"] == "append":
        s["start"] = (lens - n).contiguous()
        s["aligned"] = (s["start"] // PAGE * PAGE).contiguous()
        s["span"] = (lens - s["aligned"]).contiguous()
        mag = torch.exp(0.5 * torch.randn((B, H, 1, D), generator=g, device="cuda"))
        for name in ("k_new", "v_new"):
            # a projection's layout: tokens outermost, heads beside each other
            x = torch.randn((B, n, H, D), generator=g, device="cuda").mul_(mag.transpose(1, 2))
            s[name] = x.to(dtype).transpose(1, 2)
        s["k_out"] = torch.zeros((B, H, n + PAGE - 1, D), dtype=dtype, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
    elif c["op"] == "evict":
        w = torch.rand((pages, H, PAGE), generator=g, device="cuda")
        s["weight"] = w.mul_(w).mul_(w)
        # a share of tokens was never looked at: equal weights of zero
        s["weight"][torch.rand((pages, H, PAGE), generator=g, device="cuda") < 0.05] = 0.0
        s["pos"] = (torch.arange(PAGE, device="cuda", dtype=torch.int32)[None, None] + torch.randint(
            0, 1 << 20, (pages, H, 1), generator=g, device="cuda", dtype=torch.int32)).contiguous()
        per_to = -(-c["keep"] // PAGE)
        kind = torch.int8 if c["fmt"] == "int8" else torch.uint8
        for name in ("k", "v"):
            z = torch.zeros((B * per_to, H, PAGE, D), dtype=kind, device="cuda")
            s["to_" + name] = z if c["fmt"] == "int8" else z.view(torch.float8_e4m3fn)
            s["to_" + name + "_scale"] = torch.zeros((B * per_to, H), device="cuda")
        s["to_pos"] = torch.zeros((B * per_to, H, PAGE), dtype=torch.int32, device="cuda")
        s["to_weight"] = torch.zeros((B * per_to, H, PAGE), device="cuda")
        s["to_table"] = torch.arange(B * per_to, dtype=torch.int32, device="cuda").reshape(B, per_to)
        s["to_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros((B, H, c["keep"]), dtype=torch.int32, device="cuda")
        s["zero"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["k_out"] = torch.zeros((B, H, c["keep"], D), dtype=dtype, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
    else:
        s["q"] = torch.randn((B, n, Hq, D), generator=g, device="cuda").to(dtype).transpose(1, 2)
        s["sigma"] = 1.0 / math.sqrt(D)
        s["q_lens"] = s["q_pos"] = s["prefix"] = s["first"] = s["slopes"] = None
        if c["ragged"] and n > 1:
            s["q_lens"] = torch.randint(1, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            s["q_lens"][0] = n
            dead = torch.arange(n, device="cuda")[None, :] >= s["q_lens"][:, None]
            s["q"] = torch.where(dead[:, None, :, None], torch.full_like(s["q"], float("nan")), s["q"])
        q_lens = s["q_lens"] if s["q_lens"] is not None else torch.full((B,), n, dtype=torch.int32, device="cuda")
        last = lens
        if c["evicted"]:
            # what an eviction leaves: positions that grow along the slots, with gaps, each head its own
            step = 1 + (torch.rand((B, H, per * PAGE), generator=g, device="cuda") < 0.3).to(torch.int32)
            p = step.cumsum(2, dtype=torch.int32)
            s["pos"] = torch.zeros((pages, H, PAGE), dtype=torch.int32, device="cuda")
            at = s["table"].clamp(min=0).long()
            live = (s["table"] >= 0)[:, :, None, None]
            p = p.reshape(B, H, per, PAGE).transpose(1, 2)
            s["pos"][at[live[..., 0, 0]]] = p[live[..., 0, 0]].contiguous()
            last = (2 * lens).to(torch.int32)
            s["q_pos"] = (last - q_lens).contiguous()
        if c["prefix"]:
            s["prefix"] = torch.randint(0, c["prefix"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            s["prefix"][0] = c["prefix"]
        if c["docs"]:
            # the first token of the document that each query is in; some queries sit in none that is cached
            at = (last - q_lens)[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)[None]
            shift = torch.randint(0, c["docs"], (B, 1), generator=g, device="cuda", dtype=torch.int32)
            first = ((at + shift) // c["docs"] * c["docs"] - shift).clamp(min=0)
            none = torch.rand((B, n), generator=g, device="cuda") < 0.002
            s["first"] = torch.where(none, torch.full_like(first, 1 << 30), first).to(torch.int32).contiguous()
        if c["slopes"]:
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float32) / Hq)
        if c["op"] == "attention":
            s["out"] = torch.zeros((B, Hq, n, D), dtype=dtype, device="cuda")
            s["lse"] = torch.zeros((B, Hq, n), dtype=torch.float32, device="cuda")
        else:
            s["weight"] = torch.zeros((pages, H, PAGE), dtype=torch.float32, device="cuda")
            s["lse"] = _attention(s)[1]
    if own:
        # the descriptors and handles that a program makes once for its pools
        from bit_kv_cache_25_b200 import vq
        s["desc"] = vq.PagedDesc(H, D, c["fmt"], pages, per)
        s["cache"] = vq.PagedCache(s["desc"], k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                   pos=s["pos"], weight=s["weight"])
        if c["op"] == "evict":
            s["to_desc"] = vq.PagedDesc(H, D, c["fmt"], s["to_k"].shape[0], s["to_table"].shape[1])
            s["to_cache"] = vq.PagedCache(s["to_desc"], k=s["to_k"], v=s["to_v"], k_scale=s["to_k_scale"],
                                          v_scale=s["to_v_scale"], pos=s["to_pos"], weight=s["to_weight"])
    return s


# ---------------------------------------------------------------- plain forms
def _dense(pool, scale, table, valid, fmt):
    """[B][H][slots][D] float32 values of the sequences' pages, zero where no token is."""
    at = table.clamp(min=0).long()
    x = pool[at].float() * scale[at][..., None, None]
    x = x.transpose(1, 2).flatten(2, 3)
    return torch.where(valid[:, None, :, None], x, torch.zeros((), device="cuda"))


def _slots(pool, table):
    """[B][H][slots] of a per-slot pool."""
    return pool[table.clamp(min=0).long()].transpose(1, 2).flatten(2, 3)


def _scores(s):
    """Masked float32 scores [B][H][g][n][slots], the mask, and the shape's parts."""
    c = s["case"]
    B, H, D, n = c["batch"], c["kv_heads"], c["head_dim"], c["n"]
    grp = c["q_heads"] // H
    lens = s["lens"]
    slots = s["table"].shape[1] * PAGE
    j = torch.arange(slots, device="cuda", dtype=torch.int32)
    valid = j[None] < lens[:, None]
    k = _dense(s["k"], s["k_scale"], s["table"], valid, c["fmt"])
    q_lens = s["q_lens"] if s["q_lens"] is not None else torch.full_like(lens, n)
    i = torch.arange(n, device="cuda", dtype=torch.int32)
    live = i[None] < q_lens[:, None]                                                   # [B][n]
    q = torch.where(live[:, None, :, None], s["q"].float(), torch.zeros((), device="cuda"))
    z = (q.reshape(B, H, grp * n, D) @ k.transpose(-1, -2)).mul_(s["sigma"])
    del k
    if c["softcap"]:
        z = z.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    z = z.reshape(B, H, grp, n, slots)
    kp = _slots(s["pos"], s["table"]) if s["pos"] is not None else j.expand(B, H, slots)
    slot_i = (lens - q_lens)[:, None] + i[None]                                        # [B][n]
    if s["slopes"] is not None:
        qp = slot_i if s["q_pos"] is None else s["q_pos"][:, None] + i[None]
        far = (qp[:, None, :, None] - kp[:, :, None, :]).abs().float()                 # [B][H][n][slots]
        z.addcmul_(s["slopes"].reshape(1, H, grp, 1, 1), far[:, :, None], value=-1.0)
        del far
    see = valid[:, None, None, :] & live[:, None, :, None]
    if c["causal"]:
        past = (j[None, None] <= slot_i[:, :, None])[:, None]
        if s["prefix"] is not None:
            past = past | (kp < s["prefix"][:, None, None])[:, :, None, :]
        see = see & past
    if s["first"] is not None:
        see = see & (kp[:, :, None, :] >= s["first"][:, None, :, None])
    z.masked_fill_(~see[:, :, None], float("-inf"))
    return z, live


def _attention(s):
    c = s["case"]
    B, H, Hq, D, n = c["batch"], c["kv_heads"], c["q_heads"], c["head_dim"], c["n"]
    z, live = _scores(s)
    top = z.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top).reshape(B, Hq, n)
    p = p.div_(total.clamp(min=1e-37)).reshape(B, H, -1, p.shape[-1])
    valid = torch.arange(p.shape[-1], device="cuda")[None] < s["lens"][:, None]
    out = p @ _dense(s["v"], s["v_scale"], s["table"], valid, c["fmt"])
    return out.reshape(B, Hq, n, D), torch.where(live[:, None], lse, torch.zeros((), device="cuda"))


def _weights(s):
    c = s["case"]
    z, live = _scores(s)
    lse = s["lse"].reshape(z.shape[:-1])[..., None]
    w = z.sub_(lse.clamp(min=-3e38)).exp_().sum((2, 3))                                # [B][H][slots]
    j = torch.arange(w.shape[-1], device="cuda")
    valid = (j[None] < s["lens"][:, None])[:, None].expand_as(w)
    at = s["table"].clamp(min=0).long()
    where = ((at[:, None, :, None] * c["kv_heads"] + torch.arange(c["kv_heads"], device="cuda")[None, :, None, None]) * PAGE
             + torch.arange(PAGE, device="cuda")).flatten(2, 3)
    pool = torch.zeros_like(s["weight"])
    pool.view(-1)[where[valid]] = w[valid]
    return pool


def _round_code(x, fmt):
    """Nearest code of each value, ties to even."""
    if fmt == "int8":
        return x.round().clamp(-127, 127)
    return x.float().to(torch.float8_e4m3fn).double()


def _new_scale(amax, old, fmt):
    """The scale of a page with `amax` as its new tokens' largest value and `old` as its scale (0: none), and
    by how many powers of two it grew."""
    if fmt == "int8":
        fresh = torch.where(amax > 0, (amax.float() / 127.0).clamp(min=2.0 ** -126).double(), 0.0)
        over = amax / (127.5 * old.clamp(min=2.0 ** -140))
        m, e = torch.frexp(over)
        grow = torch.where(over < 1.0, torch.zeros_like(e), e)                          # the smallest k with over < 2^k
    else:
        m, e = torch.frexp(amax / 448.0)
        e = torch.where(m == 0.5, e - 1, e).clamp(min=-126)                             # the smallest e with amax <= 448*2^e
        fresh = torch.where(amax > 0, torch.exp2(e.double()), 0.0)
        grow = (e - torch.frexp(old.clamp(min=2.0 ** -126))[1] + 1).clamp(min=0)
    grow = torch.where((old > 0) & (amax > 0), grow, torch.zeros_like(grow))
    return torch.where(old > 0, old * torch.exp2(grow.double()), fresh), grow


def _append(s):
    c = s["case"]
    B, H, D, n = c["batch"], c["kv_heads"], c["head_dim"], c["n"]
    touched = (n + PAGE - 2) // PAGE + 1
    off = (s["start"] - s["aligned"]).long()
    first = (s["aligned"] // PAGE).long()
    slot = torch.arange(touched * PAGE, device="cuda")
    src = slot[None] - off[:, None]
    fresh = (src >= 0) & (src < n)
    index = first[:, None] + torch.arange(touched, device="cuda")[None]
    inside = index < s["table"].shape[1]
    page = s["table"].long().gather(1, index.clamp(max=s["table"].shape[1] - 1))
    live = inside & (torch.arange(touched, device="cuda")[None] * PAGE < (off + n)[:, None])
    got = []
    for x, name in ((s["k_new"], "k"), (s["v_new"], "v")):
        new = x.double().gather(2, src.clamp(0, n - 1)[:, None, :, None].expand(B, H, touched * PAGE, D))
        new = torch.where(fresh[:, None, :, None], new, 0.0).reshape(B, H, touched, PAGE, D)
        old = s[name][page[:, 0]].double()[:, :, None]                                  # [B][H][1][PAGE][D]
        amax = new.abs().amax((3, 4))                                                   # [B][H][touched]
        scale0 = torch.zeros_like(amax)
        scale0[:, :, 0] = torch.where(off[:, None] > 0, s[name + "_scale"][page[:, 0]].double(), 0.0)
        scale, grow = _new_scale(amax, scale0, c["fmt"])
        div = torch.where(scale > 0, scale, 1.0)[..., None, None]
        code = _round_code(new.div_(div), c["fmt"])
        kept = _round_code(old * torch.exp2(-grow[:, :, :1].double())[..., None, None], c["fmt"])
        code[:, :, :1] = torch.where((slot[:PAGE][None] < off[:, None])[:, None, None, :, None], kept, code[:, :, :1])
        value = (code.float() * scale.float()[..., None, None]).flatten(2, 3)[:, :, :n + PAGE - 1]
        there = slot[None, :n + PAGE - 1] < s["span"][:, None]
        got.append(torch.where(there[:, None, :, None], value, torch.zeros((), device="cuda")).to(DTYPES[c["dtype"]]))
        pool = s[name + "_scale"].clone()
        pool[page[live]] = scale.float().transpose(1, 2)[live]
        got.append(pool)
    return got


def _evict(s):
    c = s["case"]
    B, H, D, keep = c["batch"], c["kv_heads"], c["head_dim"], c["keep"]
    lens = s["lens"].long()
    slots = s["table"].shape[1] * PAGE
    j = torch.arange(slots, device="cuda")[None]
    w = _slots(s["weight"], s["table"]).double()
    w = torch.where(w.isnan(), -math.inf, w)
    safe = (j < c["sinks"]) | (j >= lens[:, None] - c["recent"])
    w = torch.where(safe[:, None], math.inf, w)
    w = torch.where((j < lens[:, None])[:, None], w, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True)[1][..., :keep]
    to_lens = lens.clamp(max=keep)
    held = (torch.arange(keep, device="cuda")[None] < to_lens[:, None])[:, None]        # [B][1][keep]
    if order.shape[-1] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=slots)
    kept = torch.where(held, order, slots).sort(-1)[0]
    kept = torch.where(held, kept, -1)
    at = kept.clamp(min=0)
    page = s["table"].clamp(min=0).long().gather(1, (at // PAGE).flatten(1)).reshape(at.shape)
    head = torch.arange(H, device="cuda")[None, :, None]
    per = s["to_table"].shape[1]
    more = per * PAGE - keep
    dest = torch.arange(keep, device="cuda")
    row = s["to_table"].long()[:, dest // PAGE]                                         # [B][keep]
    place = ((row[:, None] * H + head) * PAGE + dest % PAGE)                            # [B][H][keep]
    mask = held.expand_as(at)
    got = {"kept": kept.to(torch.int32), "lens": to_lens.to(torch.int32)}
    for name, at_rest in (("weight", s["to_weight"]), ("pos", s["to_pos"])):
        pool = torch.zeros_like(at_rest)
        pool.view(-1)[place[mask]] = s[name][page, head, at % PAGE][mask]
        got[name] = pool
    for name in ("k", "v"):
        code = s[name][page, head, at % PAGE].float().double()
        scale = torch.where(mask, s[name + "_scale"][page, head], torch.zeros((), device="cuda"))
        top = torch.nn.functional.pad(scale, (0, more)).reshape(B, H, per, PAGE).amax(-1)
        to = top.repeat_interleave(PAGE, dim=-1)[..., :keep]
        ratio = torch.where(to > 0, scale.double() / to.double(), 0.0)
        code = _round_code(code * ratio[..., None], c["fmt"])
        value = code.float() * to[..., None]
        got[name] = torch.where(mask[..., None], value, torch.zeros((), device="cuda")).to(DTYPES[c["dtype"]])
        pool = torch.zeros_like(s["to_" + name + "_scale"])
        live = torch.arange(per, device="cuda")[None] * PAGE < to_lens[:, None]
        pool[s["to_table"].long()[live]] = top.transpose(1, 2)[live]
        got[name + "_scale"] = pool
    return [got[x] for x in ("kept", "lens", "weight", "pos", "k", "k_scale", "v", "v_scale")]


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from bit_kv_cache_25_b200 import vq
        if op == "append":
            vq.vq_paged_append(s["desc"], s["cache"], s["table"], s["start"], s["k_new"], s["v_new"])
            vq.vq_paged_read(s["desc"], s["cache"], s["table"], s["aligned"], s["k_out"], s["v_out"], counts=s["span"])
            return [s["k_out"], s["k_scale"], s["v_out"], s["v_scale"]]
        if op == "evict":
            vq.vq_paged_evict(s["desc"], s["cache"], s["table"], s["lens"], s["to_desc"], s["to_cache"], s["to_table"],
                              s["to_lens"], c["keep"], sinks=c["sinks"], recent=c["recent"], kept=s["kept"])
            vq.vq_paged_read(s["to_desc"], s["to_cache"], s["to_table"], s["zero"], s["k_out"], s["v_out"],
                             counts=s["to_lens"])
            return [s["kept"], s["to_lens"], s["to_weight"], s["to_pos"], s["k_out"], s["to_k_scale"], s["v_out"],
                    s["to_v_scale"]]
        masks = dict(q_lens=s["q_lens"], q_pos=s["q_pos"], prefix=s["prefix"], first=s["first"], slopes=s["slopes"],
                     softcap=c["softcap"], causal=c["causal"])
        if op == "attention":
            vq.vq_paged_attention(s["desc"], s["cache"], s["table"], s["lens"], s["q"], s["sigma"], s["out"], s["lse"],
                                  **masks)
            return [s["out"], s["lse"]]
        vq.vq_paged_weights(s["desc"], s["cache"], s["table"], s["lens"], s["q"], s["sigma"], s["lse"],
                            accumulate=False, **masks)
        return [s["weight"]]
    if op == "append":
        return _append(s)
    if op == "evict":
        return _evict(s)
    if op == "weights":
        return [_weights(s)]
    out, lse = _attention(s)
    return [out.to(DTYPES[c["dtype"]]), lse]


# ------------------------------------------------- work and values in 64 bits
def work(case):
    """What a pass cannot do without. A ragged batch's lengths lie between a quarter of `tokens` and all of it."""
    c = case
    B, H, Hq, D, n, N = c["batch"], c["kv_heads"], c["q_heads"], c["head_dim"], c["n"], c["tokens"]
    e = 4 if c["dtype"] == "f32" else 2
    mean = N * 0.625 if c["ragged"] and B > 1 else float(N)
    if c["op"] == "append":
        return {"bytes": 2.0 * B * H * n * D * (e + 1 + e), "flops": 4.0 * B * H * n * D}
    if c["op"] == "evict":
        held = min(mean, c["keep"])
        return {"bytes": B * H * (4.0 * mean + held * (8 + 8 + 4 + 2 * D * (1 + 1 + e))), "flops": 2.0 * B * H * held * D}
    rows = n * 0.5 if c["ragged"] and n > 1 and B > 1 else float(n)
    seen = mean
    if c["causal"]:
        seen = mean - rows / 2
    if c["docs"]:
        seen = min(seen, c["docs"] / 2 if c["causal"] else mean - min(mean, c["docs"]) / 2)
    pairs = B * Hq * rows * seen
    read = B * H * (min(mean, seen + rows) if c["docs"] else mean) * D
    if c["op"] == "weights":
        return {"bytes": read + B * H * mean * 4 + B * Hq * rows * (D * e + 4), "flops": 2.0 * D * pairs}
    return {"bytes": 2.0 * read + B * Hq * rows * (2 * D * e + 4), "flops": 4.0 * D * pairs}


def _value64(raw, scale, fmt):
    """A page's values from its bytes: the codes' definition, times the scale in float32."""
    b = raw.view(torch.uint8).to(torch.int64)
    if fmt == "int8":
        code = torch.where(b > 127, b - 256, b).double()
    else:
        e, m = (b >> 3) & 15, (b & 7).double()
        mag = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2(e.double() - 10.0))
        mag = torch.where((b & 127) == 127, math.nan, mag)
        code = torch.where(b > 127, -mag, mag)
    return code, (code.float() * scale.float()).double()


def _exact_rows(s, b, h):
    """Scores of sequence b's queries for key head h: [g][q_len][len] in 64 bits, -inf where unseen, and the values."""
    c = s["case"]
    L = int(s["lens"][b])
    m = int(s["q_lens"][b]) if s["q_lens"] is not None else c["n"]
    grp = c["q_heads"] // c["kv_heads"]
    pages = s["table"][b, : -(-L // PAGE)].long()
    flat = []
    for name in ("k", "v"):
        x = _value64(s[name][pages, h], s[name + "_scale"][pages, h][:, None, None], c["fmt"])[1]
        flat.append(x.reshape(-1, c["head_dim"])[:L])
    slot = torch.arange(L, device="cuda")
    kp = s["pos"][pages, h].reshape(-1)[:L].long() if s["pos"] is not None else slot
    i = torch.arange(m, device="cuda")
    own_slot = L - m + i
    qp = own_slot if s["q_pos"] is None else int(s["q_pos"][b]) + i
    z = torch.einsum("gid,jd->gij", s["q"][b, h * grp:(h + 1) * grp, :m].double(), flat[0]) * s["sigma"]
    if c["softcap"]:
        z = c["softcap"] * torch.tanh(z / c["softcap"])
    if s["slopes"] is not None:
        z = z - s["slopes"][h * grp:(h + 1) * grp].double()[:, None, None] * (qp[:, None] - kp[None]).abs().double()
    hide = torch.zeros((m, L), dtype=torch.bool, device="cuda")
    if c["causal"]:
        hide |= slot[None] > own_slot[:, None]
        if s["prefix"] is not None:
            hide &= ~(kp[None] < int(s["prefix"][b]))
    if s["first"] is not None:
        hide |= kp[None] < s["first"][b, :m].long()[:, None]
    return z.masked_fill(hide[None], -math.inf), flat[1], pages, L, m, grp


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    B, H, Hq, D, n = c["batch"], c["kv_heads"], c["q_heads"], c["head_dim"], c["n"]
    if c["op"] in ("attention", "weights"):
        out = torch.zeros((B, Hq, n, D), dtype=torch.float64, device="cuda")
        lse = torch.zeros((B, Hq, n), dtype=torch.float64, device="cuda")
        pool = torch.zeros_like(s["weight"], dtype=torch.float64) if c["op"] == "weights" else None
        for b in range(B):
            for h in range(H):
                z, v, pages, L, m, grp = _exact_rows(s, b, h)
                own_lse = torch.logsumexp(z, -1)
                if c["op"] == "weights":
                    p = torch.exp(z - s["lse"][b, h * grp:(h + 1) * grp, :m].double().clamp(min=-1e300)[..., None])
                    w = torch.zeros(len(pages) * PAGE, dtype=torch.float64, device="cuda")
                    w[:L] = p.sum((0, 1))
                    pool[pages, h] = w.reshape(-1, PAGE)
                else:
                    p = torch.exp(z - own_lse.clamp(min=-1e300)[..., None])
                    out[b, h * grp:(h + 1) * grp, :m] = p @ v
                    lse[b, h * grp:(h + 1) * grp, :m] = own_lse
        return [pool] if c["op"] == "weights" else [out, lse]
    got = {x: torch.zeros((B, H, s["k_out"].shape[2], D), dtype=torch.float64, device="cuda") for x in ("k", "v")}
    if c["op"] == "append":
        scales = {x: s[x + "_scale"].double() for x in ("k", "v")}
        for b in range(B):
            begin = int(s["start"][b])
            for x in ("k", "v"):
                new = s[x + "_new"][b].double()                                         # [H][n][D]
                for p in range(begin // PAGE, (begin + n - 1) // PAGE + 1):
                    lo, hi = max(begin, p * PAGE), min(begin + n, (p + 1) * PAGE)
                    page = int(s["table"][b, p])
                    part = new[:, lo - begin:hi - begin]
                    before = lo - p * PAGE
                    raw, _ = _value64(s[x][page], torch.ones(1, device="cuda"), c["fmt"])
                    old = s[x + "_scale"][page].double() if before else torch.zeros(H, dtype=torch.float64, device="cuda")
                    scale, up = _grown64(part.abs().amax((1, 2)), old, c["fmt"])
                    div = torch.where(scale > 0, scale, 1.0)[:, None, None]
                    code = torch.cat([_nearest64(raw[:, :before] * (2.0 ** -up)[:, None, None], c["fmt"]),
                                      _nearest64(part / div, c["fmt"])], 1)
                    at = p * PAGE - begin // PAGE * PAGE
                    got[x][b, :, at:at + code.shape[1]] = code * scale[:, None, None]
                    scales[x][page] = scale
        return [got["k"], scales["k"], got["v"], scales["v"]]
    pools = {x: torch.zeros_like(s["to_" + x], dtype=torch.float64) for x in ("weight", "k_scale", "v_scale")}
    for b in range(B):
        L = int(s["lens"][b])
        pages = s["table"][b, : -(-L // PAGE)].long()
        for h in range(H):
            w = s["weight"][pages, h].reshape(-1)[:L].double().cpu()
            hold = min(L, c["keep"])
            safe = torch.zeros(L, dtype=torch.bool)
            safe[:c["sinks"]] = True
            safe[max(0, L - c["recent"]):] = True
            if L > c["keep"]:
                rest = torch.nonzero(~safe).reshape(-1)
                best = rest[torch.argsort(w[rest], descending=True, stable=True)[:hold - int(safe.sum())]]
                safe[best] = True
                at = torch.nonzero(safe).reshape(-1).cuda()
            else:
                at = torch.arange(L, device="cuda")
            per = -(-hold // PAGE)
            to = s["to_table"][b, :per].long()
            gap = (0, per * PAGE - hold)
            src, place = pages[at // PAGE], at % PAGE
            pools["weight"][to, h] = torch.nn.functional.pad(s["weight"][src, h, place].double(), gap).reshape(per, PAGE)
            for x in ("k", "v"):
                scale = s[x + "_scale"][src, h].double()
                code, _ = _value64(s[x][src, h, place], torch.ones(1, device="cuda"), c["fmt"])
                top = torch.nn.functional.pad(scale, gap).reshape(per, PAGE).amax(1)
                pools[x + "_scale"][to, h] = top
                top = top[torch.arange(hold, device="cuda") // PAGE, None]
                new = _nearest64(code * scale[:, None] / torch.where(top > 0, top, 1.0), c["fmt"])
                got[x][b, h, :hold] = new * top
    return [None, None, pools["weight"], None, got["k"], pools["k_scale"], got["v"], pools["v_scale"]]


def _nearest64(x, fmt):
    """The nearest code's value: whole numbers, or e4m3's grid, ties to even."""
    if fmt == "int8":
        return torch.round(x).clamp(-127, 127)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(-6, 8)
    # log2 next to a power of two: the grid's exponent from the value itself
    e = torch.where(x.abs() >= torch.exp2(e + 1), e + 1, torch.where((x.abs() < torch.exp2(e)) & (e > -6), e - 1, e))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _grown64(amax, old, fmt):
    """A page's scale after new tokens up to amax, and the powers of two that it grew by."""
    scale, up = old.clone(), torch.zeros_like(old)
    for t in range(len(old)):
        a, o = float(amax[t]), float(old[t])
        if o == 0:
            if fmt == "int8":
                one = float((torch.tensor(a, dtype=torch.float32) / 127.0)) if a > 0 else 0.0
                scale[t] = max(one, 2.0 ** -126) if a > 0 else 0.0
            else:
                e = -126
                while a > 448.0 * 2.0 ** e:
                    e += 1
                scale[t] = 2.0 ** e if a > 0 else 0.0
            continue
        k = 0
        while (a >= 127.5 * o * 2.0 ** k) if fmt == "int8" else (a > 448.0 * o * 2.0 ** k):
            k += 1
        scale[t], up[t] = o * 2.0 ** k, k
    return scale, up
