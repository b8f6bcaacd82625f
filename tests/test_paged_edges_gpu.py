"""Paged 8-bit cache on the GPU at the edges of what the calls allow: references that
move in every page, against the oracle with the bounds of test_paged_gpu.py."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as po
from bit_kv_cache_25_b200 import vq
from test_paged_gpu import Paged, _q

pytestmark = pytest.mark.gpu


def _rising(D, fmt, pages, step, n, dtype, G=1):
    """A cache whose scores rise by `step` nats from page to page, and queries for it (softmax scale 1)."""
    p = Paged(1, 1, D, fmt, pages, seed=pages)
    p.fill([pages * 64 - 5])
    for j in range(pages):
        page = p.table[0, j]
        c = p.g.integers(-3, 4, (64, D)).astype(np.float64)
        c[:, 0] = np.copysign(96.0, step)  # (a scale is never negative)
        p.o["k"][page, 0] = po.encode(c, fmt)
        p.o["k_scale"][page, 0] = abs(step) / 96.0 * (j + 1)
    p.push()
    q = _q(p, G, n, dtype, 0.02)
    q[..., 0] = 1.0
    return p, q


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G,pages", [(60, 1, 9), (130, 1, 6), (150, 2, 9)])
def test_a_reference_that_moves_in_every_page(n, G, pages, D, fmt, dtype):
    """Each page's best score passes the one before by more than 8 in log2, so both pages of every key tile move the
    row's reference, and what the first of them stored is rescaled by the second."""
    p, q = _rising(D, fmt, pages, 6.5, n, dtype, G)
    p.attend(q, 1.0)


@pytest.mark.parametrize("scales", ["tiny_first", "huge_first", "zeros", "mixed"])
@pytest.mark.parametrize("n,dtype,D", [(1, torch.bfloat16, 128), (20, torch.float16, 64), (60, torch.bfloat16, 64),
                                       (150, torch.bfloat16, 128), (150, torch.float16, 64), (300, torch.bfloat16, 128)])
def test_v_scales_that_lie_far_apart(n, dtype, D, scales):
    """Pages whose V differ by up to 2^215 and pages of zeros, in one sequence, seen together (whole rows) and apart
    (causal rows and windows that see one kind of page only), with scores that favour either kind."""
    p = Paged(2, 1, D, "int8", 6, seed=n)
    p.fill([384, max(n, 200)])
    power = {"tiny_first": [-120, -118, 0, 2, -3, 1], "huge_first": [90, 88, -5, 3, -100, 0],
             "zeros": [None, None, -3, None, 4, None], "mixed": [0, -60, None, -119, 95, 20]}[scales]
    if dtype == torch.float16:  # (whose outputs end at 65504: the largest scale is an ordinary one)
        power = [e if e is None else e - max(x for x in power if x is not None) for e in power]
        power = [e if e is None else max(e, -119) for e in power]
    for b in range(2):
        for j, e in enumerate(power):
            page = p.table[b, j]
            if e is None:
                p.o["v"][page], p.o["v_scale"][page] = 0, 0.0
            else:
                p.o["v_scale"][page] *= 2.0 ** e
    p.push()
    q = _q(p, 2, n, dtype)
    for scale in (0.05, 0.6):
        p.attend(q, scale, causal=True)
        p.attend(q, scale)
    first = np.minimum(p.g.integers(0, 384, (2, n)), (p.lens - n)[:, None] + np.arange(n)[None]).astype(np.int32)
    p.attend(q, 0.3, causal=True, first=first)


@pytest.mark.parametrize("n", [1, 150])
def test_the_largest_and_smallest_v(n):
    """V as large as vq.h allows (times the tokens seen 2^112), and down to scales of 2^-126."""
    for e in (103, -119):
        p = Paged(1, 1, 64, "int8", 4, seed=n)
        p.fill([200])
        x = p.g.normal(size=p.o["v_scale"].shape)
        p.o["v_scale"][...] = np.maximum(np.exp(0.3 * x) * 2.0 ** (e - 7), 2.0 ** -126)
        p.push()
        p.attend(_q(p, 4, n, torch.bfloat16), 0.3, causal=n > 1)


@pytest.mark.parametrize("n", [1, 20, 150])
def test_a_bad_page_among_very_low_scores(n):
    """Tokens of a page id out of range count as unseen, also where every score that is seen lies far below 0."""
    p, q = _rising(64, "int8", 4, -150.0, n, torch.bfloat16)
    for bad in (0, 1, 3):
        table = p.dtable.clone()
        table[0, bad] = -1
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
        vq.vq_paged_attention(p.desc, p.cache, table, p.dev(p.lens), q, 1.0, out, lse)
        torch.cuda.synchronize()
        assert vq.vq_poll_device_error() == 4
        k, v = (x.astype(np.float64) for x in po.read(p.o, p.table, 0, 0, 0, int(p.lens[0])))
        keep = [j for j in range(int(p.lens[0])) if j // 64 != bad]
        z = q[0, 0].double().cpu().numpy() @ k[keep].T
        want, wlse, w = po.attention(z, v[keep])
        # the score's float32 error at this size (products of 64 channels, z to log2 units and back), weights to fp16
        dz = np.abs(z).max() * (64 + 16 + 8) * 2.0 ** -24
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * dz + 2.0 ** -19) * (w @ np.abs(v[keep])) + 1e-6
        assert (np.abs(out[0, 0].double().cpu().numpy() - want) <= tol).all(), bad
        assert (np.abs(lse[0, 0].double().cpu().numpy() - wlse) <= 2 * dz + np.abs(wlse) * 2.0 ** -22 + 1e-4).all(), bad


@pytest.mark.parametrize("cap", [1.0, 50.0, 1e3, 1e4, 1e6])
@pytest.mark.parametrize("n,G,pos", [(1, 4, False), (9, 2, True), (60, 1, False), (130, 2, True)])
def test_a_cap_of_any_size_is_exact_for_scores_far_below_it(cap, n, G, pos, monkeypatch):
    """Scores of a few units under caps up to 1e6: close to no cap. One key far below the others (beyond a quarter of
    the cap) must not cost the others their bits."""
    scores = po.scores

    def without_the_far_ones(*a, **kw):
        z, err = scores(*a, **kw)  # (a key 200 below the row's best has no weight, whatever its score's error)
        return z, np.where(z < z.max(1, keepdims=True) - 200.0, 0.0, err)

    monkeypatch.setattr(po, "scores", without_the_far_ones)
    for low in (False, True):
        p = Paged(1, 2, 64, "int8", 5, seed=n)
        p.fill([300])
        if low:
            page = p.table[0, 1]
            for name in ("k", "v"):
                p.o[name][page] = po.encode(p.g.integers(-2, 3, p.o[name][page].shape).astype(np.float64), "int8")
            p.o["k"][page, :, 5, 0] = po.encode(np.array(-127.0), "int8")
            p.o["k_scale"][page] = np.float32(cap / 127)  # channel 0 of that key: -cap, of the other keys +-2 / 127 cap
            p.o["k"][page, :, :5, 0] = 0
            p.o["k"][page, :, 6:, 0] = 0
        p.push()
        q = _q(p, 2 * G, n, torch.bfloat16, 0.5)
        if low:
            q[..., 0] = 1.0
            q[..., 1:] *= min(1.0, 100.0 / cap)
        m = dict(slopes=2.0 ** -np.arange(1, 2 * G + 1), causal=True, prefix=[70]) if pos else {}
        p.attend(q, 0.4, softcap=cap, **m)


def test_evicted_codes_whose_quotient_is_a_tie():
    """Tokens of pages of scale 15 join a page of scale 22 (times a power of two): 11 * 15 / 22 = 7.5 exactly, and so on:
    to the even code."""
    for num, den in ((15, 22), (5, 26), (7, 38), (21, 22), (125, 254), (3, 2 ** 20 + 2)):
        p = Paged(1, 1, 64, "int8", 2, seed=num)
        p.lens = np.array([128], np.int32)
        p.o["k"][...] = p.o["v"][...] = 0
        codes = np.concatenate([np.arange(-127, 128), [0]]).astype(np.int8).view(np.uint8).reshape(4, 64)
        for n in ("k", "v"):
            p.o[n][p.table[0, 0], 0, :4] = codes
            p.o[n + "_scale"][...] = np.float32(num * 2.0 ** -9)
            p.o[n + "_scale"][p.table[0, 1]] = np.float32(den * 2.0 ** -9)
        p.o["weight"][...] = 0
        p.o["weight"][p.table[0, 0], 0, :4] = 1
        p.o["weight"][p.table[0, 1], 0, 7] = 1
        p.push()
        to = Paged(1, 1, 64, "int8", 1, seed=1)
        kept, to_lens = torch.zeros((1, 1, 5), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        vq.vq_paged_evict(p.desc, p.cache, p.dtable, p.dev(p.lens), to.desc, to.cache, to.dtable, to_lens, 5, kept=kept)
        po.evict(p.o, p.table, p.lens, to.o, to.table, 5, 0, 0)
        assert kept.tolist() == [[[0, 1, 2, 3, 71]]]
        to.check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [4, 20, 150])
def test_weights_of_queries_of_any_content(n, causal):
    """A live query of NaN or infinity that sees nothing gives no weight to anything; one that sees some tokens spoils
    those and leaves what it does not see alone."""
    L = 250 if causal else 640  # (causal or not: tiles of keys that only some rows see, or all but those that see nothing)
    p = Paged(1, 2, 64, "int8", 10, seed=n, pos=False)
    p.fill([L])
    q = _q(p, 4, n, torch.bfloat16)
    first = np.zeros((1, n), np.int32)
    first[0, 1] = 2 ** 30          # sees nothing
    first[0, 2] = L - n            # sees the call's own tokens, its first three where causal
    args = dict(first=p.dev(first), causal=causal)

    def weights(q):
        out, lse = torch.zeros_like(q), torch.zeros((1, 4, n), device="cuda")
        vq.vq_paged_attention(p.desc, p.cache, p.dtable, p.dev(p.lens), q, 0.125, out, lse, **args)
        vq.vq_paged_weights(p.desc, p.cache, p.dtable, p.dev(p.lens), q, 0.125, lse, accumulate=False, **args)
        torch.cuda.synchronize()
        assert vq.vq_poll_device_error() == 0
        return np.array([po.per_slot({"weight": p.cache.weight.cpu().numpy()}, "weight", p.table, 0, h, L) for h in range(2)]), lse

    good, lse = weights(q)
    assert torch.isneginf(lse[0, :, 1]).all() and np.isfinite(good).all()
    for bad in (float("nan"), float("inf"), float("-inf")):
        x = q.clone()
        x[0, :, 1] = bad
        got, _ = weights(x)
        assert np.array_equal(got, good), bad
        x[0, :2, 2] = bad          # key head 0's queries
        got, lse = weights(x)
        assert torch.isnan(lse[0, :2, 2]).all() and np.array_equal(got[1], good[1])
        hit = np.zeros(L, bool)
        hit[L - n:L - n + 3 if causal else L] = True
        assert np.isnan(got[0][hit]).all() and np.array_equal(got[0][~hit], good[0][~hit]), bad


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_of_scales_whose_half_is_not_a_float(dtype):
    """Scales just above 2^-126 with an odd last bit: quotients next to a half go to their nearest code."""
    p = Paged(1, 1, 64, "int8", 8, seed=3)
    for j in range(8):
        s = 2.0 ** -126 + (2 * j + 1) * 2.0 ** -149
        x = np.float64(np.arange(-64, 64)[:, None] * s)
        x = np.rint((x + 0.5 * s) / 2.0 ** -149) + p.g.integers(-1, 2, x.shape)
        x = np.concatenate([x.reshape(2, 64) * 2.0 ** -149, np.zeros((62, 64))]).astype(np.float32)
        x[2, 0] = np.float32(127 * s)
        t = torch.from_numpy(x)[None, None].cuda().to(dtype)
        p.append(t, t)
    p.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_sequences_that_share_pages(fmt):
    """A common prefix of two pages, one of them with other pages behind it: read, attended and evicted from by all;
    weights by one call after the other, which sum up."""
    p = Paged(3, 2, 64, fmt, 6, seed=21, pos=False, weight=False)
    p.table[1, :2] = p.table[2, :2] = p.table[0, :2]
    p.dtable = p.dev(p.table)
    p.fill([300, 200, 131])
    x = [torch.zeros((3, 2, 128, 64), device="cuda") for _ in range(2)]
    vq.vq_paged_read(p.desc, p.cache, p.dtable, p.dev(np.zeros(3, np.int32)), *x)
    for b in range(3):
        for h in range(2):
            assert np.array_equal(x[0][b, h].cpu().numpy(), po.read(p.o, p.table, 0, h, 0, 128)[0])
    for n in (1, 20, 60, 150):
        p.attend(_q(p, 4, n, torch.bfloat16), 0.125, causal=True)
    # what each appends behind the prefix is its own
    p.append(*p.tokens(40))
    p.check()
    p.attend(_q(p, 4, 3, torch.bfloat16), 0.125, causal=True)

    cache = vq.PagedCache(p.desc, k=p.cache.k, v=p.cache.v, k_scale=p.cache.k_scale, v_scale=p.cache.v_scale,
                          weight=torch.zeros(p.cache.k.shape[:3], device="cuda"))
    for n in (2, 60):
        q = _q(p, 4, n, torch.bfloat16)
        lens, out, lse = p.dev(p.lens), torch.zeros_like(q), torch.zeros((3, 4, n), device="cuda")
        vq.vq_paged_attention(p.desc, p.cache, p.dtable, lens, q, 0.125, out, lse, causal=True)
        cache.weight.zero_()
        for b in range(3):
            i = slice(b, b + 1)
            vq.vq_paged_weights(p.desc, cache, p.dtable[i], lens[i], q[i], 0.125, lse[i], causal=True)
        got = cache.weight.cpu().numpy()
        w, wt = p.expect(q, 0.125, np.full(3, n), causal=True)[4:]
        want, tol = np.zeros(got.shape), np.zeros(got.shape)
        for b in range(3):
            for h in range(2):
                for j in range(int(p.lens[b])):
                    at = p.table[b, j // 64], h, j % 64
                    want[at] += w[b][h][j]
                    tol[at] += wt[b][h][j]
        assert (np.abs(got - want) <= tol + np.abs(want) * 2.0 ** -22).all()
    p.cache = cache
    p.o["weight"] = got
    keep = 100
    to = Paged(3, 2, 64, fmt, 2, seed=22)
    kept, to_lens = torch.zeros((3, 2, keep), dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    vq.vq_paged_evict(p.desc, p.cache, p.dtable, p.dev(p.lens), to.desc, to.cache, to.dtable, to_lens, keep, sinks=2, recent=7, kept=kept)
    want, _ = po.evict(p.o, p.table, p.lens, to.o, to.table, keep, 2, 7)
    assert np.array_equal(kept.cpu().numpy(), want)
    to.check()


@pytest.mark.parametrize("n,G,pos", [(1, 4, False), (20, 2, True), (60, 1, False), (150, 2, True), (150, 1, False)])
def test_a_lower_bound_without_a_causal_mask_hides_nothing_behind(n, G, pos):
    """`first` alone is a lower bound: what lies behind a query is seen to the sequence's end."""
    p = Paged(2, 2, 64, "int8", 5, seed=n, pos=pos)
    p.fill([320, max(n, 131)])
    first = p.g.integers(0, 320, (2, n)).astype(np.int32)
    p.attend(_q(p, 2 * G, n, torch.bfloat16, 2.0), 0.125, first=first)


@pytest.mark.parametrize("n", [1, 20, 150])
def test_queries_with_one_channel_far_above_the_others(n, monkeypatch):
    """bf16 query rows with a channel 2^30 above the others: what lies 2^-24 and more below a row's largest magnitude is
    exact only to 2^-32 of that magnitude (half of fp16's smallest step under the row's power of two)."""
    p = Paged(1, 2, 64, "int8", 4, seed=n)
    p.fill([250])
    for j in range(4):
        page = p.o["k"][p.table[0, j]]
        page[..., 0] = po.encode(np.where(p.g.random(page.shape[:-1]) < 0.5, 0.0, 1.0), "int8")
    p.push()
    scores = po.scores

    def with_the_rounding_of_queries(c, table, b, h, hq, length, q, sigma, **kw):
        z, err = scores(c, table, b, h, hq, length, q, sigma, **kw)
        k = np.abs(po.read(c, table, b, h, 0, length)[0].astype(np.float64))
        return z, err + sigma * np.abs(q).max(1, keepdims=True) * 2.0 ** -32 * k.sum(1)[None]

    monkeypatch.setattr(po, "scores", with_the_rounding_of_queries)
    for up in (20, 23, 30):
        q = _q(p, 4, n, torch.bfloat16)
        q[..., 0] = 2.0 ** up
        p.attend(q, 2.0 ** -up)
        p.attend(q, 2.0 ** -max(up - 8, 0) * 0.01)


def test_evict_more_tokens_than_shared_memory_has_keys_for():
    """Sequences of more than 49152 tokens: the later keys are gathered again for every digit."""
    L, keep, H = 49152 + 3000, 20000, 2
    pages = -(-L // 64)
    for kind in ("distinct", "ties"):
        p = Paged(2, H, 64, "int8", pages, seed=2, pos=False)
        p.lens = np.array([L, 49153], np.int32)
        w = p.o["weight"]
        w[...] = p.g.gamma(0.1, size=w.shape) if kind == "distinct" else p.g.choice(np.array([0.0, 0.5, 2.0], np.float32), w.shape)
        for n in ("k_scale", "v_scale"):
            p.o[n][...] = 0.5
        p.push()
        to = Paged(2, H, 64, "int8", -(-keep // 64), seed=3)
        kept, to_lens = torch.zeros((2, H, keep), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
        vq.vq_paged_evict(p.desc, p.cache, p.dtable, p.dev(p.lens), to.desc, to.cache, to.dtable, to_lens, keep, sinks=5,
                          recent=100, kept=kept)
        torch.cuda.synchronize()
        assert vq.vq_poll_device_error() == 0 and to_lens.tolist() == [keep, keep]
        for b in range(2):
            n = int(p.lens[b])
            for h in range(H):
                flat = w[p.table[b], h].reshape(-1)[:n].astype(np.float64)
                flat[:5] = flat[n - 100:] = np.inf
                want = np.sort(np.lexsort((np.arange(n), -flat))[:keep])
                assert np.array_equal(kept[b, h].cpu().numpy(), want)
                at = to.table[b][np.arange(keep) // 64]
                got = to.cache.weight[torch.from_numpy(at).cuda().long(), h, torch.arange(keep, device="cuda") % 64].cpu().numpy()
                assert np.array_equal(got, w[p.table[b][want // 64], h, want % 64])


def test_two_calls_at_once_on_streams_that_waited():
    """Two calls that run together, each on a stream that waits for its inputs and for the outputs' first contents."""
    p = Paged(2, 4, 128, "int8", 64, seed=17)
    p.fill([4096, 2000])
    lens = p.dev(p.lens)
    qs = [_q(p, 16, n, torch.bfloat16) for n in (1, 3, 40)]
    want = []
    for q in qs:
        out = torch.zeros_like(q)
        vq.vq_paged_attention(p.desc, p.cache, p.dtable, lens, q, 0.1, out)
        want.append(out)
    outs = [[torch.zeros_like(q) for _ in range(10)] for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(10):
        for s, q, o in zip(streams, qs, outs):
            vq.vq_paged_attention(p.desc, p.cache, p.dtable, lens, q, 0.1, o[i], stream=s)
    torch.cuda.synchronize()
    assert vq.vq_poll_device_error() == 0
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


@pytest.mark.parametrize("n", [1, 20, 60, 150])
def test_queries_of_broadcast_heads_and_sequences_without_tokens(n):
    """Query views whose batch and head strides are 0, a sequence of no token, negative slopes."""
    p = Paged(3, 2, 128, "e4m3", 3, seed=n)
    p.fill([192, 0, 77])
    x = _q(p, 1, n, torch.float16)[:1]
    p.attend(x.expand(3, 6, n, 128), 0.09)
    p.attend(x.expand(3, 6, n, 128), 0.09, causal=True, slopes=-2.0 ** -np.arange(4, 10))


def test_captured_without_a_workspace():
    """Graphs whose calls take their workspace from the allocator, replayed in turn and between other allocations."""
    p = Paged(2, 2, 128, "int8", 100, seed=31)
    p.fill([6400, 3001])
    lens = p.dev(p.lens)
    graphs = []
    for n in (1, 6, 40):
        q = _q(p, 4, n, torch.bfloat16)
        assert vq.vq_paged_attention_workspace(p.desc, 2, 4, n) > 0
        want, out = torch.zeros_like(q), torch.zeros_like(q)
        vq.vq_paged_attention(p.desc, p.cache, p.dtable, lens, q, 0.1, want, causal=True)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            vq.vq_paged_attention(p.desc, p.cache, p.dtable, lens, q, 0.1, out, causal=True)
            vq.vq_paged_attention(p.desc, p.cache, p.dtable, lens, q, 0.1, out, causal=True)
        graphs.append((g, q, want, out))  # (q stays alive: the graph reads it)
    for _ in range(3):
        for g, _, want, out in graphs:
            out.fill_(7.0)
            junk = torch.full((1 << 22,), 9.0, device="cuda")
            g.replay()
            junk = junk + 1
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    assert vq.vq_poll_device_error() == 0
    del graphs


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n,G", [(1, 1), (4, 2), (9, 1), (16, 1), (6, 2), (2, 5), (16, 3), (64, 1), (70, 2)])
def test_a_distance_bias_by_positions_under_masks_by_slots(n, G, fmt, D, dtype, causal):
    """Positions with gaps for the bias, and no mask that needs them; what lies behind the last token is not seen."""
    p = Paged(2, 2, D, fmt, 3, seed=n)
    p.fill([max(n, 36), max(n, 131)])
    for b in range(2):
        for h in range(2):
            run = np.cumsum(p.g.integers(1, 4, 192))
            for j in range(3):
                p.o["pos"][p.table[b, j], h] = run[64 * j:64 * j + 64]
    p.push()
    for slopes, cap in ((2.0 ** -np.linspace(3, 9, 2 * G), 0.0), (-2.0 ** -np.linspace(3, 9, 2 * G), 5.0)):
        p.attend(_q(p, 2 * G, n, dtype), 0.1, causal=causal, slopes=slopes, q_pos=[100, 400], softcap=cap)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_of_signed_zeros_and_nan_alone(fmt, dtype):
    """Nothing but zeros of both signs and NaN: a scale of 0 and codes of +0, also when later tokens bring values."""
    p = Paged(1, 2, 64, fmt, 2, seed=2)
    x = torch.zeros((1, 2, 9, 64), device="cuda", dtype=dtype)
    x[..., ::2] = -0.0
    x[:, :, 3, 5] = float("nan")
    p.append(x, -x)
    p.check()
    p.append(*p.tokens(3, dtype))
    p.append(x, -x)
    p.check()
