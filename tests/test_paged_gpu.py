"""Paged 8-bit cache on the GPU against the oracle: codes, scales, positions and
kept slots to the bit, attention and weights within bounds that follow from the
arithmetic.

The bound of an output element: its rounding, u * |out|, u half a step relative to
the value (bf16 2^-8, fp16 2^-11); and what a relative error of each weight makes
of sum w |v|: 2^-11 for its rounding to fp16 (and 2^-31 per key for weights below
fp16's smallest normal number), twice the float32 error of its score, and 2^-19 for
exponentials, factors and sums in float32. Log-sum-exp: the score's error and the
float32 error of a sum of so many terms."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as po
from bit_kv_cache_25_b200 import vq

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# Half of the type's smallest step: what rounding is off by below its smallest normal number. (fp16's steps
# there are 2^-24: where one token of value 0 takes all but 7e-8 of a row's weight, the row's sum of 2.9e-8 is
# rounded to 0, which is 2^-25 off at most, and that is more than 2^-11 of it.)
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


class Paged:
    """A cache with its block table on the device, and the oracle's copy."""

    def __init__(self, B, H, D, fmt, max_pages, seed=0, spare=3, pos=True, weight=True):
        g = np.random.default_rng(seed)
        self.g, self.B, self.H, self.D, self.fmt = g, B, H, D, fmt
        pages = B * max_pages + spare
        self.desc = vq.PagedDesc(H, D, fmt, pages, max_pages)
        order = g.permutation(pages)
        self.table = order[:B * max_pages].reshape(B, max_pages).astype(np.int32)
        # every byte that no token has been written to: NaN codes, NaN scales
        shape = (pages, H, 64)
        self.o = {"k": np.full(shape + (D,), 0x7F, np.uint8), "v": np.full(shape + (D,), 0x7F, np.uint8),
                  "k_scale": np.full((pages, H), np.nan, np.float32), "v_scale": np.full((pages, H), np.nan, np.float32),
                  "pos": np.full(shape, -7, np.int32) if pos else None,
                  "weight": np.full(shape, 9.0, np.float32) if weight else None, "fmt": fmt}
        self.cache = vq.PagedCache(self.desc, **{n: None if a is None else torch.from_numpy(a.copy()).cuda()
                                                 for n, a in self.o.items() if n != "fmt"})
        self.dtable = torch.from_numpy(self.table).cuda()
        self.lens = np.zeros(B, np.int32)

    def dev(self, a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    def append(self, k, v, counts=None, pos=None, oracle=True):
        n = k.shape[2]
        cnt = np.full(self.B, n, np.int32) if counts is None else np.asarray(counts, np.int32)
        vq.vq_paged_append(self.desc, self.cache, self.dtable, self.dev(self.lens), k, v,
                           counts=None if counts is None else self.dev(cnt),
                           pos=None if pos is None else self.dev(np.asarray(pos, np.int32)))
        if oracle:
            po.append(self.o, self.table, self.lens, cnt, k.float().cpu().numpy(), v.float().cpu().numpy(), pos)
        self.lens = self.lens + cnt

    def check(self):
        torch.cuda.synchronize()
        assert vq.vq_poll_device_error() == 0
        for n in ("k", "v"):
            off = getattr(self.cache, n).view(torch.uint8).cpu().numpy() != self.o[n]
            assert not off.any(), (n, np.argwhere(off)[:5].tolist())
        for n in ("k_scale", "v_scale", "pos", "weight"):
            if self.o[n] is not None:
                assert np.array_equal(getattr(self.cache, n).cpu().numpy(), self.o[n], equal_nan=n != "pos"), n

    def tokens(self, n, dtype=torch.bfloat16, spread=0.0):
        """New K, V in a projection's layout, [B][n][H][D] transposed."""
        out = []
        for _ in range(2):
            x = self.g.normal(size=(self.B, n, self.H, self.D)) * np.exp(spread * self.g.normal(size=(self.B, n, 1, 1)))
            x[..., :3] *= 20
            out.append(torch.from_numpy(x.astype(np.float32)).to(dtype).cuda().transpose(1, 2))
        return out

    def fill(self, lens):
        """Sequences of these lengths, without going through append."""
        o, g = self.o, self.g
        for b, L in enumerate(lens):
            for j in range(-(-int(L) // 64)):
                page, used = self.table[b, j], min(64, int(L) - 64 * j)
                for n in ("k", "v"):
                    c = np.clip(g.normal(size=(self.H, used, self.D)) * 30, -127, 127)
                    o[n][page, :, :used] = po.encode(c, self.fmt)
                    s = np.exp(g.normal(size=self.H)) * 0.02
                    o[n + "_scale"][page] = s if self.fmt == "int8" else 2.0 ** np.floor(np.log2(s))
                if o["pos"] is not None:
                    o["pos"][page, :, :used] = np.arange(64 * j, 64 * j + used)
        self.lens = np.asarray(lens, np.int32)
        self.push()

    def push(self):
        for n, a in self.o.items():
            if n != "fmt" and a is not None:
                t = getattr(self.cache, n)
                (t.view(torch.uint8) if n in ("k", "v") else t).copy_(torch.from_numpy(a))

    def expect(self, q, sigma, q_lens, **m):
        """Oracle's out, lse, their bounds, per-token weights and their bounds."""
        B, Hq, n, D = q.shape
        G = Hq // self.H
        qn = q.float().cpu().numpy().astype(np.float64)
        out, lse = np.zeros(q.shape), np.zeros((B, Hq, n))
        tol, ltol = np.zeros(q.shape), np.zeros((B, Hq, n))
        w = [[None] * self.H for _ in range(B)]
        wt = [[None] * self.H for _ in range(B)]
        for b in range(B):
            L, ql = int(self.lens[b]), int(q_lens[b])
            for h in range(self.H):
                v = po.read(self.o, self.table, b, h, 0, L)[1].astype(np.float64)
                w[b][h], wt[b][h] = np.zeros(L), np.zeros(L)
                for hq in range(h * G, (h + 1) * G):
                    z, err = po.scores(
                        self.o, self.table, b, h, hq, L, qn[b, hq, :ql], sigma, q_len=ql,
                        q_pos=None if m.get("q_pos") is None else int(m["q_pos"][b]),
                        prefix=0 if m.get("prefix") is None else int(m["prefix"][b]),
                        first=None if m.get("first") is None else m["first"][b],
                        slope=0.0 if m.get("slopes") is None else float(m["slopes"][hq]), cap=m.get("softcap", 0.0),
                        causal=m.get("causal", False))
                    o_, l_, w_ = po.attention(z, v)
                    out[b, hq, :ql], lse[b, hq, :ql] = o_, l_
                    dz = np.where(np.isfinite(z), err, 0).max(1) if L else np.zeros(ql)
                    each = 2.0 ** -11 + 2 * dz + 2.0 ** -19
                    top = w_.max(1) if L else np.zeros(ql)
                    tol[b, hq, :ql] = (HALF[q.dtype] * np.abs(o_) + each[:, None] * (w_ @ np.abs(v))
                                       + (top * 2.0 ** -31)[:, None] * np.abs(v).sum(0)[None] + TINY[q.dtype])
                    ltol[b, hq, :ql] = 2 * dz + 2.0 ** -20 + (L / 8 + 64) * 2.0 ** -24 + np.abs(np.where(np.isfinite(l_), l_, 0)) * 2.0 ** -22
                    w[b][h] += w_.sum(0)
                    wt[b][h] += (w_ * (4 * dz + 2.0 ** -18 + ql * G * 2.0 ** -24 + np.abs(np.where(np.isfinite(l_), l_, 0)) * 2.0 ** -22)[:, None]).sum(0) + 1e-36
        return out, lse, tol, ltol, w, wt

    def attend(self, q, sigma, q_lens=None, **m):
        """Attention and weights on the GPU, checked against the oracle; returns what the call left."""
        B, Hq, n, D = q.shape
        ql = np.full(B, n, np.int32) if q_lens is None else np.asarray(q_lens, np.int32)
        args = {k: self.dev(np.asarray(v, np.float32 if k == "slopes" else np.int32)) if isinstance(v, (list, np.ndarray)) else v
                for k, v in m.items() if v is not None}
        if q_lens is not None:
            args["q_lens"] = self.dev(ql)
        # outputs inside a larger tensor, tokens outermost; what is not a live row must stay as it is
        room = torch.full((B, n + 1, Hq + 1, D), 77.0, dtype=q.dtype, device="cuda")
        out = room[:, :n, :Hq].transpose(1, 2)
        lse = torch.full((B, Hq, n), 55.0, device="cuda")
        vq.vq_paged_attention(self.desc, self.cache, self.dtable, self.dev(self.lens), q, sigma, out, lse, **args)
        torch.cuda.synchronize()
        assert vq.vq_poll_device_error() == 0
        want, wlse, tol, ltol, w, wt = self.expect(q, sigma, ql, **m)
        live = np.arange(n)[None, None, :] < ql[:, None, None]
        got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(B):
            assert (got[b, :, ql[b]:] == 77.0).all() and (glse[b, :, ql[b]:] == 55.0).all()
        assert (room[:, n:] == 77.0).all() and (room[:, :, Hq:] == 77.0).all()
        bad = ~(np.abs(got - want) <= tol)
        bad &= np.broadcast_to(live[..., None], bad.shape)
        assert not bad.any(), ((np.abs(got - want) / np.maximum(tol, 1e-300))[bad].max(), np.argwhere(bad)[:4].tolist(), bad.sum())
        seen = np.isfinite(wlse)
        livef = np.broadcast_to(live, seen.shape)
        assert np.array_equal(np.isneginf(glse) & livef, ~seen & livef)
        assert (np.abs(np.where(seen & livef, glse - np.where(seen, wlse, 0), 0)) <= ltol).all(), "lse"
        if self.o["weight"] is not None:
            before = self.o["weight"].copy()
            for acc in (False, True):
                vq.vq_paged_weights(self.desc, self.cache, self.dtable, self.dev(self.lens), q, sigma, lse, accumulate=acc, **args)
            torch.cuda.synchronize()
            assert vq.vq_poll_device_error() == 0
            gw = self.cache.weight.cpu().numpy()
            touched = np.zeros(gw.shape, bool)
            for b in range(B):
                for h in range(self.H):
                    for j in range(int(self.lens[b])):
                        at = (self.table[b, j // 64], h, j % 64)
                        touched[at] = True
                        assert abs(gw[at] - 2 * w[b][h][j]) <= 2 * wt[b][h][j] + abs(w[b][h][j]) * 2.0 ** -23, (b, h, j)
            assert np.array_equal(gw[~touched], before[~touched])
            self.o["weight"] = gw.copy()
        return out, lse


def _q(p, Hq, n, dtype, scale=1.0):
    x = p.g.normal(size=(p.B, n, Hq, p.D)).astype(np.float32) * scale
    return torch.from_numpy(x).to(dtype).cuda().transpose(1, 2)


# ------------------------------------------------------------------- append, read
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_append_to_the_bit(fmt, D, dtype):
    p = Paged(2, 3, D, fmt, 6, seed=D)
    for n in (1, 1, 5, 64, 1, 130, 63):
        p.append(*p.tokens(n, dtype, spread=1.5))
    p.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_token_by_token_with_growing_values(fmt):
    p = Paged(1, 2, 64, fmt, 2, seed=5)
    for t in range(70):
        k, v = p.tokens(1, torch.float32)
        p.append(k * 2.0 ** (t % 23 - 9), v * 1.07 ** t, pos=[1000 + 3 * t])
    p.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_ragged_counts_and_rows_not_read(fmt):
    p = Paged(4, 1, 64, fmt, 4, seed=6)
    p.append(*p.tokens(7))
    k, v = p.tokens(100)
    for b, c in enumerate((0, 1, 57, 100)):
        k[b, :, c:] = float("nan")
        v[b, :, c:] = float("inf")
    p.append(k, v, counts=[0, 1, 57, 100])
    p.append(*p.tokens(3))
    p.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_special_values(fmt):
    """Zeros, signed zeros, subnormals, infinities, NaN, the largest and the exact half-way quotients."""
    p = Paged(1, 1, 64, fmt, 16, seed=7)
    f = np.float32
    nan, inf = np.nan, np.inf
    pages = [np.zeros(64), np.full(64, -0.0), np.full(64, 1e-45), f(1e-39) * np.arange(64),
             np.where(np.arange(64) == 5, nan, np.arange(64) - 32.0), np.where(np.arange(64) == 9, inf, 1.0),
             np.full(64, nan), np.where(np.arange(64) == 1, -inf, nan), np.full(64, 3.4e38),
             np.concatenate([[127.0], np.arange(63) + 0.5]), np.concatenate([[-448.0], np.arange(63) * 0.28125 * 2.0 ** -6]),
             np.concatenate([[254.0], (np.arange(63) + 0.5) * 2 * (1 + 2.0 ** -23)]),
             np.concatenate([[12.7], f(0.1) * (np.arange(63) + f(0.5))])]
    for row in pages:  # each its own page: 64 tokens, 64 channels, the row rolled so that every channel sees it
        x = np.stack([np.roll(row, t) for t in range(64)]).astype(f)[None, None]
        t = torch.from_numpy(x).cuda()
        p.append(t, t)
    k = torch.zeros((1, 1, 5, 64), device="cuda")
    p.append(k, k)                 # a page of zeros so far
    p.append(k + 3.0, k - 2.5)     # its first values
    p.append(k, k + 1e30)          # and a growth past every older code
    p.check()


def test_append_borders_of_growth():
    for fmt, most in (("int8", 127.5), ("e4m3", 448.0)):
        p = Paged(1, 1, 64, fmt, 1, seed=8)
        one = torch.ones((1, 1, 1, 64), device="cuda")
        p.append(one * (127.0 if fmt == "int8" else 448.0), one)
        for x in (np.nextafter(np.float32(most), np.float32(0)), np.float32(most), np.nextafter(np.float32(most), np.float32(1e9))):
            p.append(one * float(x), one * float(x))
        p.check()


def test_append_of_broadcast_heads_and_aliased_batch():
    p = Paged(3, 4, 64, "int8", 2, seed=9)
    x = torch.randn((1, 1, 70, 64), device="cuda", dtype=torch.bfloat16)
    p.append(x.expand(3, 4, 70, 64), x.expand(3, 4, 70, 64))
    p.check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_read(fmt, D, dtype):
    p = Paged(3, 2, D, fmt, 4, seed=10)
    p.fill([256, 130, 1])
    start, counts = np.array([60, 0, 0], np.int32), np.array([150, 130, 0], np.int32)
    out = [torch.full((3, 150, 2, D), 5.0, dtype=dtype, device="cuda").transpose(1, 2) for _ in range(2)]
    vq.vq_paged_read(p.desc, p.cache, p.dtable, p.dev(start), out[0], out[1], counts=p.dev(counts))
    torch.cuda.synchronize()
    assert vq.vq_poll_device_error() == 0
    for b in range(3):
        for h in range(2):
            want = po.read(p.o, p.table, b, h, int(start[b]), int(start[b] + counts[b]))
            for t in range(2):
                assert torch.equal(out[t][b, h, :counts[b]].cpu(), torch.from_numpy(want[t]).to(dtype).reshape(-1, D))
                assert (out[t][b, h, counts[b]:] == 5.0).all()


# --------------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_single_token(fmt, D, dtype, G):
    p = Paged(5, 2, D, fmt, 8, seed=G)
    p.fill([512, 1, 0, 65, 333])
    p.attend(_q(p, 2 * G, 1, dtype), D ** -0.5)


@pytest.mark.parametrize("lens", [[1], [31], [32], [33], [63], [64], [65], [127], [128], [129], [200]])
def test_lengths_around_a_page(lens):
    p = Paged(1, 1, 64, "e4m3", 4, seed=lens[0])
    p.fill(lens)
    p.attend(_q(p, 4, 1, torch.bfloat16), 0.125)


@pytest.mark.parametrize("fmt,dtype,D", [("int8", torch.bfloat16, 128), ("e4m3", torch.float16, 64)])
@pytest.mark.parametrize("n,G", [(2, 1), (5, 2), (17, 1), (33, 4), (130, 1), (129, 2), (300, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_chunks(fmt, dtype, D, n, G, causal):
    p = Paged(2, 2, D, fmt, 6, seed=n)
    p.fill([n + 57, 384 if n <= 384 else n])
    p.attend(_q(p, 2 * G, n, dtype), D ** -0.5, causal=causal)


@pytest.mark.parametrize("n,G", [(1, 4), (9, 2), (140, 2)])
@pytest.mark.parametrize("fmt,dtype,D", [("int8", torch.float16, 64), ("e4m3", torch.bfloat16, 128)])
@pytest.mark.parametrize("masks", ["cap", "slopes", "prefix", "first", "all", "all_pos"])
def test_masks_and_biases(masks, fmt, dtype, D, n, G):
    p = Paged(3, 2, D, fmt, 5, seed=n, pos=masks == "all_pos")
    p.fill([320, n, max(n, 131)])
    m = dict(causal=True)
    every = masks.startswith("all")
    if masks == "cap" or every:
        m["softcap"] = 2.5
    if masks == "slopes" or every:
        m["slopes"] = 2.0 ** -np.arange(1, 2 * G + 1)
    if masks == "prefix" or every:
        m["prefix"] = [77, 1 << 30, 0]
    if masks == "first" or every:
        first = p.g.integers(-5, 320, (3, n)).astype(np.int32)
        first[0, 0] = 2 ** 31 - 1     # a query that sees nothing
        first[1, :] = -2 ** 31
        m["first"] = first
    if masks == "all_pos":
        step = p.g.integers(1, 4, p.o["pos"].shape[0] * 0 + 5 * 64)
        for b in range(3):
            run = np.cumsum(step)
            for j in range(5):
                p.o["pos"][p.table[b, j]] = run[64 * j:64 * j + 64]
        p.push()
        m["q_pos"] = [700, 3, 900]
    p.attend(_q(p, 2 * G, n, dtype, 3.0), D ** -0.5, **m)


@pytest.mark.parametrize("n,G", [(7, 1), (40, 2), (150, 1)])
def test_padded_queries_of_any_content(n, G):
    p = Paged(4, 2, 64, "e4m3", 4, seed=n)
    ql = np.array([n, 1, 0, n // 2], np.int32)
    p.fill([256, 1, 100, max(n // 2, 3)])
    q = _q(p, 2 * G, n, torch.bfloat16)
    for b in range(4):
        q[b, :, ql[b]:] = float("nan")
    p.attend(q, 0.125, q_lens=ql, causal=True)
    p.attend(q, 0.125, q_lens=ql)


@pytest.mark.parametrize("rows", [8, 9, 16, 17, 47, 48, 49, 128, 129, 256, 257])
def test_rows_around_the_kernels_tiles(rows):
    p = Paged(2, 1, 128, "int8", 7, seed=rows)
    p.fill([rows + 100, 448])
    p.attend(_q(p, 1, rows, torch.bfloat16), 0.09, causal=True)


@pytest.mark.parametrize("n", [3, 140])
def test_more_queries_than_tokens_leaves_rows_empty(n):
    p = Paged(2, 1, 64, "int8", 2, seed=n)
    p.fill([2, 70])
    p.attend(_q(p, 2, n, torch.float16), 0.125, causal=True)
    p.attend(_q(p, 2, n, torch.float16), 0.125, causal=True, prefix=[1, 5])


@pytest.mark.parametrize("n", [1, 5, 200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_peaked_and_far_apart_values(n, dtype):
    """Scores hundreds apart, pages whose V differ by 2^20, queries of tiny and large magnitude."""
    p = Paged(2, 2, 128, "int8", 5, seed=n)
    p.fill([320, 257])
    for b in range(2):
        for j in range(5):
            p.o["v_scale"][p.table[b, j]] *= 2.0 ** (5 * j - 10)
            p.o["k_scale"][p.table[b, j]] *= 3.0 ** j
    p.push()
    q = _q(p, 4, n, dtype)
    q[:, 0] *= 6
    q[:, 1] *= 2.0 ** -13
    p.attend(q, 0.3)


def test_a_nan_or_infinite_query_stays_in_its_row():
    for n in (4, 200):
        p = Paged(1, 1, 64, "int8", 4, seed=3)
        p.fill([250])
        q = _q(p, 2, n, torch.bfloat16)
        good = p.attend(q.clone(), 0.125)[0].clone()
        p.cache.weight.zero_()
        q[0, 0, 1] = float("nan")
        q[0, 1, 2, 0] = float("inf")
        out = torch.zeros_like(good)
        lse = torch.zeros((1, 2, n), device="cuda")
        vq.vq_paged_attention(p.desc, p.cache, p.dtable, p.dev(p.lens), q, 0.125, out, lse)
        hit = torch.zeros((1, 2, n), dtype=torch.bool, device="cuda")
        hit[0, 0, 1] = hit[0, 1, 2] = True
        assert torch.equal(out[~hit], good[~hit])
        assert not torch.isfinite(out[0, 0, 1]).any() and not torch.isfinite(out[0, 1, 2]).any()


@pytest.mark.parametrize("n,G,pages", [(1, 4, 400), (1, 16, 120), (3, 5, 90), (60, 1, 90), (3, 64, 70), (130, 2, 70)])
@pytest.mark.parametrize("masks", ["plain", "all"])
def test_a_long_axis_is_split_and_joined(n, G, pages, masks):
    """One sequence and one head: its pages go to many CTAs, some of them with nothing to see."""
    D = 64 if n == 3 else 128
    p = Paged(1, 1, D, "e4m3" if G > 2 else "int8", pages, seed=pages + n, weight=pages < 400)
    p.fill([pages * 64 - 29])
    m = {}
    if masks == "all":
        first = p.g.integers(0, pages * 64, (1, n)).astype(np.int32)
        first[0, 0] = pages * 64 - 100
        m = dict(causal=True, softcap=20.0, slopes=2.0 ** -np.linspace(4, 12, G), prefix=[500], first=first)
    p.attend(_q(p, G, n, torch.bfloat16, 2.0), D ** -0.5, **m)


def test_repeats_to_the_bit_on_streams_and_with_a_workspace():
    p = Paged(3, 2, 128, "e4m3", 40, seed=4)
    p.fill([2500, 64, 1111])
    for n in (1, 6, 150):
        q = _q(p, 8, n, torch.bfloat16)
        lens = p.dev(p.lens)
        size = vq.vq_paged_attention_workspace(p.desc, 3, 8, n)
        ref = None
        side = torch.cuda.Stream()
        for kind in ("plain", "workspace", "stream", "handle"):
            out, lse = torch.zeros_like(q), torch.zeros((3, 8, n), device="cuda")
            side.wait_stream(torch.cuda.current_stream())
            kw = {"plain": {}, "workspace": dict(workspace=torch.full((size + 16,), 255, dtype=torch.uint8, device="cuda")),
                  "stream": dict(stream=side), "handle": dict(stream=side.cuda_stream)}[kind]
            vq.vq_paged_attention(p.desc, p.cache, p.dtable, lens, q, 0.1, out, lse, causal=True, **kw)
            side.synchronize()
            torch.cuda.synchronize()
            if ref is None:
                ref = out.clone(), lse.clone()
            assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1]), (n, kind)
        if size:
            with pytest.raises(vq.VqError, match="workspace"):
                vq.vq_paged_attention(p.desc, p.cache, p.dtable, lens, q, 0.1, out, lse,
                                      workspace=torch.empty(size - 1, dtype=torch.uint8, device="cuda"))
    assert vq.vq_poll_device_error() == 0


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes, the sequences in its last pages."""
    H, D, pages = 8, 128, 66000
    desc = vq.PagedDesc(H, D, "int8", pages, 3)
    cache = vq.PagedCache(desc, weights=True, positions=True)
    assert cache.k.numel() > 2 ** 32
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((1, H, 170, D), generator=g, device="cuda") for _ in range(2))
    zero, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([170], dtype=torch.int32, device="cuda")
    vq.vq_paged_append(desc, cache, table, zero, k, v)
    kd, vd = torch.zeros_like(k), torch.zeros_like(v)
    vq.vq_paged_read(desc, cache, table, zero, kd, vd)
    assert (kd - k).abs().max() < 0.03 and (vd - v).abs().max() < 0.03
    for n in (1, 140):
        q = torch.randn((1, H, n, D), generator=g, device="cuda").to(torch.float16)
        out, lse = torch.zeros_like(q), torch.zeros((1, H, n), device="cuda")
        vq.vq_paged_attention(desc, cache, table, lens, q, 0.1, out, lse)
        z = (q.double() @ kd.double().transpose(2, 3)) * 0.1
        w = torch.softmax(z, -1)
        bound = 2.0 ** -11 * (w @ vd.double()).abs() + 2.0 ** -10 * (w @ vd.double().abs())
        assert ((out.double() - w @ vd.double()).abs() <= bound).all()
        vq.vq_paged_weights(desc, cache, table, lens, q, 0.1, lse, accumulate=False)
        got = cache.weight[table[0].long()].transpose(0, 1).reshape(H, -1)[:, :170]
        assert torch.allclose(got.double(), w.sum(2)[0], rtol=2.0 ** -14, atol=0)
    kept, to_lens = torch.zeros((1, H, 64), dtype=torch.int32, device="cuda"), zero.clone()
    to_table = torch.tensor([[pages - 9]], dtype=torch.int32, device="cuda")
    to_desc = vq.PagedDesc(H, D, "int8", pages, 1)
    to = vq.PagedCache(to_desc, k=cache.k, v=cache.v, k_scale=cache.k_scale, v_scale=cache.v_scale, pos=cache.pos, weight=cache.weight)
    vq.vq_paged_evict(desc, cache, table, lens, to_desc, to, to_table, to_lens, 64, kept=kept)
    want = torch.sort(torch.sort(got, dim=-1, descending=True, stable=True)[1][:, :64])[0]
    assert torch.equal(kept[0].long(), want) and int(to_lens) == 64
    assert torch.equal(cache.pos[pages - 9].long(), want) and vq.vq_poll_device_error() == 0


# ---------------------------------------------------------------------- eviction
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (64, 0, 0), (65, 4, 16), (200, 0, 200), (200, 200, 0), (130, 1, 100), (400, 3, 3)])
def test_evict_to_the_bit(fmt, D, keep, sinks, recent):
    p = Paged(4, 2, D, fmt, 6, seed=keep)
    p.fill([384, keep, 0, min(384, keep + 1)] if keep <= 384 else [384, 100, 0, 1])
    w = p.o["weight"]
    w[...] = p.g.choice(np.array([0.0, -0.0, 0.5, 0.25, 1e-30, 1e-45, -3.0, np.inf, -np.inf, np.nan], np.float32), w.shape)
    p.push()
    to = Paged(4, 2, D, fmt, -(-keep // 64), seed=keep + 1)
    kept, to_lens = torch.full((4, 2, keep), -5, dtype=torch.int32, device="cuda"), torch.full((4,), -5, dtype=torch.int32, device="cuda")
    vq.vq_paged_evict(p.desc, p.cache, p.dtable, p.dev(p.lens), to.desc, to.cache, to.dtable, to_lens, keep, sinks=sinks,
                      recent=recent, kept=kept)
    want, lens = po.evict(p.o, p.table, p.lens, to.o, to.table, keep, sinks, recent)
    assert np.array_equal(kept.cpu().numpy(), want) and np.array_equal(to_lens.cpu().numpy(), lens)
    to.check()
    p.check()


def test_evict_many_distinct_weights():
    p = Paged(1, 3, 64, "int8", 160, seed=1, pos=False)
    p.lens = np.array([160 * 64 - 17], np.int32)
    p.o["weight"][...] = p.g.gamma(0.1, size=p.o["weight"].shape)
    p.push()
    keep = 3000
    to = Paged(1, 3, 64, "int8", 47, seed=2)
    kept, to_lens = torch.zeros((1, 3, keep), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    vq.vq_paged_evict(p.desc, p.cache, p.dtable, p.dev(p.lens), to.desc, to.cache, to.dtable, to_lens, keep, sinks=5, recent=100, kept=kept)
    torch.cuda.synchronize()
    for h in range(3):
        w = po.per_slot(p.o, "weight", p.table, 0, h, int(p.lens[0]))
        assert kept[0, h].tolist() == po.keep_slots(w, int(p.lens[0]), keep, 5, 100)
    assert vq.vq_poll_device_error() == 0


# ------------------------------------------------------------ together, and bad input
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_run_of_them(fmt):
    """Prompt, weights, single tokens, eviction, single tokens on what was kept."""
    D, Hq = 64, 4
    p = Paged(2, 2, D, fmt, 5, seed=12)
    p.append(*p.tokens(150), counts=[150, 90])
    slopes = 2.0 ** -np.arange(1, Hq + 1)
    p.o["weight"][...] = 0
    p.push()
    p.attend(_q(p, Hq, 150, torch.bfloat16), 0.125, q_lens=[150, 90], causal=True, slopes=slopes)
    for _ in range(3):
        p.append(*p.tokens(1))
        p.attend(_q(p, Hq, 1, torch.bfloat16), 0.125, causal=True, slopes=slopes)
    seen = p.lens.copy()
    to = Paged(2, 2, D, fmt, 3, seed=13)
    kept, to_lens = torch.zeros((2, 2, 100), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    vq.vq_paged_evict(p.desc, p.cache, p.dtable, p.dev(p.lens), to.desc, to.cache, to.dtable, to_lens, 100, sinks=2, recent=10, kept=kept)
    want, lens = po.evict(p.o, p.table, p.lens, to.o, to.table, 100, 2, 10)
    assert np.array_equal(kept.cpu().numpy(), want)
    to.lens = lens.astype(np.int32)
    to.check()
    for i in range(4):
        to.append(*to.tokens(1), pos=seen + i)
        to.attend(_q(to, Hq, 1, torch.bfloat16), 0.125, causal=True, slopes=slopes, q_pos=list(seen + i), softcap=20.0)


def _flag():
    torch.cuda.synchronize()
    return vq.vq_poll_device_error()


def test_bad_pages_and_lengths_are_skipped_and_flagged():
    p = Paged(3, 1, 64, "int8", 4, seed=14)
    p.fill([200, 200, 200])
    q = _q(p, 2, 1, torch.bfloat16)
    good = p.attend(q, 0.125)[0].clone()
    # sequence 1: its second page is out of range: the same as if those tokens were masked
    table = p.dtable.clone()
    for bad in (-1, p.desc.num_pages, 2 ** 31 - 1, -2 ** 31):
        table[1, 1] = bad
        for n in (1, 150):
            qq = q.expand(3, 2, n, 64).contiguous()
            out, lse = torch.zeros_like(qq), torch.zeros((3, 2, n), device="cuda")
            vq.vq_paged_attention(p.desc, p.cache, table, p.dev(p.lens), qq, 0.125, out, lse)
            assert _flag() == 4
            o = dict(p.o)
            keep = [j for j in range(200) if not 64 <= j < 128]
            k, v = po.read(o, p.table, 1, 0, 0, 200)
            z = 0.125 * (q[1, :, 0].double().cpu().numpy() @ k[keep].astype(np.float64).T)
            want = po.attention(z, v[keep].astype(np.float64))[0]
            assert np.abs(out[1, :, -1].double().cpu().numpy() - want).max() <= 2.0 ** -6 * np.abs(want).max()
            if n == 1:
                assert torch.equal(out[[0, 2]], good[[0, 2]])
            vq.vq_paged_weights(p.desc, p.cache, table, p.dev(p.lens), qq, 0.125, lse)
            assert _flag() == 4
    # lengths out of range
    for n in (1, 150):
        qq = q.expand(3, 2, n, 64).contiguous()
        out, lse = torch.zeros_like(qq), torch.zeros((3, 2, n), device="cuda")
        lens = torch.tensor([-1, 4 * 64 + 1, 200], dtype=torch.int32, device="cuda")
        vq.vq_paged_attention(p.desc, p.cache, p.dtable, lens, qq, 0.125, out, lse)
        assert _flag() == 4 and (out[0] == 0).all() and torch.isneginf(lse[0]).all()
        ql = torch.tensor([n, n + 1, -1], dtype=torch.int32, device="cuda")
        vq.vq_paged_attention(p.desc, p.cache, p.dtable, p.dev(p.lens), qq, 0.125, out, lse, q_lens=ql)
        assert _flag() == 4
    # appends and reads past the table, at negative starts, into bad pages: nothing written
    before = p.cache.k.clone(), p.cache.v.clone(), p.cache.k_scale.clone()
    x = torch.randn((3, 1, 2, 64), device="cuda")
    start = torch.tensor([256, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    vq.vq_paged_append(p.desc, p.cache, p.dtable, start, x, x)
    assert _flag() == 4
    y = torch.full_like(x, 3.0)
    vq.vq_paged_read(p.desc, p.cache, p.dtable, start, y, y.clone())
    assert _flag() == 4 and (y == 3.0).all()
    table[:, 3] = torch.tensor([-1, p.desc.num_pages, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    vq.vq_paged_append(p.desc, p.cache, table, torch.full((3,), 200, dtype=torch.int32, device="cuda"), x, x)
    assert _flag() == 4
    for a, b in zip(before, (p.cache.k, p.cache.v, p.cache.k_scale)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # eviction from and into bad pages
    to = Paged(3, 1, 64, "int8", 2, seed=15)
    kept, to_lens = torch.zeros((3, 1, 100), dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    bad_to = to.dtable.clone()
    bad_to[2, 0] = 10 ** 9
    vq.vq_paged_evict(p.desc, p.cache, table, p.dev(p.lens), to.desc, to.cache, bad_to, to_lens, 100, kept=kept)
    assert _flag() == 4 and to_lens.tolist() == [100, 100, 100]
    assert not any(64 <= j < 128 for j in kept[1, 0].tolist())


def test_captured_and_replayed():
    """A decoding step in a CUDA graph, replayed as the lengths grow; two graphs that share one workspace in turn."""
    B, H, D, Hq = 3, 2, 128, 8
    a, b = (Paged(B, H, D, "int8", 6, seed=16) for _ in range(2))
    for p in (a, b):
        p.append(*p.tokens(100, spread=0.5), counts=[100, 3, 64])
    size = max(16, vq.vq_paged_attention_workspace(a.desc, B, Hq, 1))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    steps = [a.tokens(1) + [_q(a, Hq, 1, torch.bfloat16)] for _ in range(4)]

    def step(p, k, v, q, lens, out, lse, w):
        vq.vq_paged_append(p.desc, p.cache, p.dtable, lens, k, v)
        lens.add_(1)
        vq.vq_paged_attention(p.desc, p.cache, p.dtable, lens, q, 0.1, out, lse, workspace=w)
        vq.vq_paged_weights(p.desc, p.cache, p.dtable, lens, q, 0.1, lse)

    want = []
    la = a.dev(a.lens)
    for k, v, q in steps:
        out, lse = torch.zeros_like(q), torch.zeros((B, Hq, 1), device="cuda")
        step(a, k, v, q, la, out, lse, None)
        want.append((out, lse))
    lb = b.dev(b.lens)
    k, v, q = (torch.zeros_like(t) for t in steps[0])
    graphs = []
    keep = lb.clone(), *(t.clone() for t in (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale, b.cache.pos, b.cache.weight))
    side = torch.cuda.Stream()
    for _ in range(2):
        out, lse = torch.zeros_like(q), torch.zeros((B, Hq, 1), device="cuda")
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            step(b, k, v, q, lb, out, lse, ws)
        graphs.append((g, out, lse))
    for t, s in zip((lb, b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale, b.cache.pos, b.cache.weight), keep):
        t.copy_(s)
    for i, (sk, sv, sq) in enumerate(steps):
        for t, s in zip((k, v, q), (sk, sv, sq)):
            t.copy_(s)
        g, out, lse = graphs[i % 2]
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    assert torch.equal(a.cache.weight, b.cache.weight) and torch.equal(a.cache.k, b.cache.k)
    assert vq.vq_poll_device_error() == 0
    del graphs


def test_two_calls_at_once_on_two_streams():
    p = Paged(2, 4, 128, "int8", 64, seed=17)
    p.fill([4096, 2000])
    lens = p.dev(p.lens)
    qs = [_q(p, 16, n, torch.bfloat16) for n in (1, 3)]
    want = []
    for q in qs:
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
        vq.vq_paged_attention(p.desc, p.cache, p.dtable, lens, q, 0.1, out, lse)
        want.append(out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [[torch.zeros_like(q) for _ in range(10)] for q in qs]
    for i in range(10):
        for s, q, o in zip(streams, qs, outs):
            vq.vq_paged_attention(p.desc, p.cache, p.dtable, lens, q, 0.1, o[i], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)
