"""The paged cache's entry points refuse bad arguments on the host, before any
launch (no GPU): the C ABI with a status, the binding with ValueError."""
import ctypes

import pytest
import torch

from bit_kv_cache_25_b200 import vq

BAD = 0x1000  # never dereferenced: validation fails first
INV, UNS, MIS = vq.VQ_ERR_INVALID_ARGUMENT, vq.VQ_ERR_UNSUPPORTED, vq.VQ_ERR_MISALIGNED
ST = (ctypes.c_int64 * 3)(3 * 4 * 64, 4 * 64, 64)


def _desc(**kw):
    a = dict(kv_heads=3, head_dim=64, code=0, num_pages=8, max_pages=4)
    a.update(kw)
    return vq.vq_paged_desc(*a.values())


def _cache(**kw):
    a = dict(k=BAD, v=BAD, k_scale=BAD, v_scale=BAD, pos=None, weight=BAD)
    a.update(kw)
    return vq.vq_paged_cache(*a.values())


def _query(**kw):
    q = vq.vq_paged_query(2, 6, 4, vq.VQ_BF16, BAD, ST, BAD, BAD, None, None, None, None, None, 0.125, 0.0, 0)
    for k, v in kw.items():
        setattr(q, k, (ctypes.c_int64 * 3)(*v) if k == "q_strides" else v)
    return q


BAD_DESCS = [(dict(kv_heads=0), INV), (dict(num_pages=0), INV), (dict(max_pages=0), INV), (dict(head_dim=96), UNS),
             (dict(code=2), UNS), (dict(code=-1), UNS), (dict(max_pages=(1 << 24) + 1), UNS),
             (dict(num_pages=(1 << 31) - 1, kv_heads=64), UNS)]
BAD_CACHES = [(dict(k=None), INV), (dict(v_scale=None), INV), (dict(v=BAD + 8), MIS), (dict(k_scale=BAD + 4), MIS),
              (dict(pos=BAD + 4), MIS), (dict(weight=BAD + 8), MIS)]


def _append(d=None, c=None, batch=2, n=4, k=BAD, v=BAD, dtype=0, ks=ST, vs=ST, table=BAD, start=BAD, counts=None, pos=None):
    return vq.raw_lib().vq_paged_append(ctypes.byref(d or _desc()), ctypes.byref(c or _cache()), batch, n, k, v, dtype, ks,
                                        vs, table, start, counts, pos, None)


def _read(d=None, c=None, batch=2, n=4, table=BAD, start=BAD, counts=None, k=BAD, v=BAD, dtype=0, ks=ST, vs=ST):
    return vq.raw_lib().vq_paged_read(ctypes.byref(d or _desc()), ctypes.byref(c or _cache()), batch, n, table, start,
                                      counts, k, v, dtype, ks, vs, None)


def _attention(d=None, c=None, q=None, out=BAD, os=ST, lse=None, ws=None, size=0):
    return vq.raw_lib().vq_paged_attention(ctypes.byref(d or _desc()), ctypes.byref(c or _cache()),
                                           ctypes.byref(q or _query()), out, os, lse, ws, size, None)


def _weights(d=None, c=None, q=None, lse=BAD, acc=1):
    return vq.raw_lib().vq_paged_weights(ctypes.byref(d or _desc()), ctypes.byref(c or _cache()),
                                         ctypes.byref(q or _query()), lse, acc, None)


def _evict(d=None, c=None, batch=2, table=BAD, lens=BAD, td=None, tc=None, to_table=BAD, to_lens=BAD + 64, keep=64, sinks=0,
           recent=0, kept=BAD):
    return vq.raw_lib().vq_paged_evict(ctypes.byref(d or _desc()), ctypes.byref(c or _cache()), batch, table, lens,
                                       ctypes.byref(td or _desc()), ctypes.byref(tc or _cache()), to_table, to_lens, keep,
                                       sinks, recent, kept, None)


@pytest.mark.parametrize("call", [_append, _read, _attention, _weights, _evict])
def test_bad_descriptors_and_pools(call):
    for kw, st in BAD_DESCS:
        assert call(d=_desc(**kw)) == st, kw
        assert vq.raw_lib().vq_last_error()
    for kw, st in BAD_CACHES:
        assert call(c=_cache(**kw)) == st, kw


@pytest.mark.parametrize("call", [_append, _read])
def test_bad_token_calls(call):
    strided = (ctypes.c_int64 * 3)(3 * 4 * 64, 4 * 64, 60)
    negative = (ctypes.c_int64 * 3)(-64, 4 * 64, 64)
    for kw, st in [(dict(batch=0), INV), (dict(n=0), INV), (dict(k=None), INV), (dict(v=None), INV),
                   (dict(k=BAD + 8), MIS), (dict(dtype=3), UNS), (dict(ks=strided), MIS), (dict(vs=negative), INV),
                   (dict(table=None), INV), (dict(start=None), INV), (dict(start=BAD + 2), MIS),
                   (dict(counts=BAD + 1), MIS), (dict(batch=1 << 30, n=1 << 30), UNS)]:
        assert call(**kw) == st, kw


def test_outputs_without_a_zero_stride():
    zero = (ctypes.c_int64 * 3)(3 * 4 * 64, 0, 64)
    assert _read(ks=zero) == INV and _attention(os=zero) == INV


@pytest.mark.parametrize("call", [_attention, _weights])
def test_bad_queries(call):
    nan, inf = float("nan"), float("inf")
    for kw, st in [(dict(batch=0), INV), (dict(n=0), INV), (dict(q_heads=0), INV), (dict(q_heads=5), INV), (dict(q=None), INV),
                   (dict(q=BAD + 2), MIS), (dict(dtype=vq.VQ_F32), UNS), (dict(dtype=9), UNS),
                   (dict(q_strides=(64, 64, 63)), MIS), (dict(block_table=None), INV), (dict(lens=None), INV),
                   (dict(lens=BAD + 2), MIS), (dict(q_lens=BAD + 1), MIS), (dict(first=BAD + 2), MIS),
                   (dict(slopes=BAD + 2), MIS), (dict(softmax_scale=0.0), INV), (dict(softmax_scale=nan), INV),
                   (dict(softmax_scale=inf), INV), (dict(softcap=-1.0), INV), (dict(softcap=nan), INV),
                   (dict(softcap=1e-9), INV), (dict(causal=2), INV), (dict(prefix=BAD), INV),
                   (dict(n=1 << 30), UNS)]:
        assert call(q=_query(**kw)) == st, kw


def test_bad_attention_and_weights_outputs():
    assert _attention(out=None) == INV and _attention(out=BAD + 8) == MIS
    assert _attention(lse=BAD + 4) == MIS and _attention(ws=BAD + 8, size=1 << 20) == MIS
    assert _weights(lse=None) == INV and _weights(lse=BAD + 4) == MIS and _weights(acc=2) == INV
    assert _weights(c=_cache(weight=None)) == INV


def test_bad_evictions():
    for kw, st in [(dict(batch=0), INV), (dict(table=None), INV), (dict(lens=None), INV), (dict(to_table=None), INV),
                   (dict(to_lens=BAD + 2), MIS), (dict(to_lens=BAD), INV), (dict(to_lens=BAD + 4), INV), (dict(kept=None), INV), (dict(kept=BAD + 2), MIS), (dict(keep=0), INV),
                   (dict(sinks=-1), INV), (dict(recent=-1), INV), (dict(sinks=40, recent=25), INV),
                   (dict(keep=4 * 64 + 1), INV), (dict(td=_desc(kv_heads=2)), INV), (dict(td=_desc(head_dim=128)), INV),
                   (dict(td=_desc(code=1)), INV), (dict(c=_cache(weight=None)), INV), (dict(tc=_cache(k=None)), INV),
                   (dict(keep=2 ** 31 - 1, td=_desc(max_pages=1)), INV)]:
        assert _evict(**kw) == st, kw


def test_null_structures():
    lib = vq.raw_lib()
    d, c, q = _desc(), _cache(), _query()
    assert lib.vq_paged_attention(None, ctypes.byref(c), ctypes.byref(q), BAD, ST, None, None, 0, None) == INV
    assert lib.vq_paged_attention(ctypes.byref(d), None, ctypes.byref(q), BAD, ST, None, None, 0, None) == INV
    assert lib.vq_paged_attention(ctypes.byref(d), ctypes.byref(c), None, BAD, ST, None, None, 0, None) == INV
    assert lib.vq_paged_attention(ctypes.byref(d), ctypes.byref(c), ctypes.byref(q), BAD, None, None, None, 0, None) == INV
    assert lib.vq_paged_attention_workspace(ctypes.byref(d), 2, 6, 4, None) == INV


# ---- the binding
def _pool(**kw):
    desc = vq.PagedDesc(3, 64, "int8", 8, 4)
    return desc, vq.PagedCache(desc, device="cpu", positions=True, weights=True, **kw)


def test_binding_refuses_pools_that_do_not_fit():
    desc = vq.PagedDesc(3, 64, "e4m3", 8, 4)
    with pytest.raises(ValueError, match="int8"):
        vq.PagedDesc(3, 64, "e5m2", 8, 4)
    with pytest.raises(ValueError, match="dtype"):
        vq.PagedCache(desc, k=torch.zeros(8, 3, 64, 64, dtype=torch.int8))
    with pytest.raises(ValueError, match="shape"):
        vq.PagedCache(desc, k=torch.zeros(8, 3, 32, 64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="shape"):
        vq.PagedCache(desc, k_scale=torch.zeros(3, 8).t())
    with pytest.raises(AttributeError):
        vq.PagedCache(desc, device="cpu").k = None


def test_binding_refuses_host_tensors_and_other_descriptors():
    desc, cache = _pool()
    x = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    ints = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        vq.vq_paged_append(desc, cache, table, ints, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        vq.vq_paged_attention(desc, cache, table, ints, x, 0.1, x)
    with pytest.raises(ValueError, match="another descriptor"):
        vq.vq_paged_read(vq.PagedDesc(3, 64, "int8", 8, 5), cache, table, ints, x, x)


def test_binding_refuses_arrays_that_do_not_fit(monkeypatch):
    desc, cache = _pool()
    monkeypatch.setattr(vq, "_paged_cache_check", lambda d, c: -1)
    x = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    ints = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 4, dtype=torch.int32)
    good = dict(block_table=table, start=ints, k=x, v=x)
    for kw, msg in [(dict(block_table=table[:, :3]), "shape"), (dict(block_table=table.long()), "int64"),
                    (dict(start=ints[:1]), "shape"), (dict(start=None), "missing"), (dict(k=x[:, :2], v=x[:, :2]), "shape"),
                    (dict(v=x.float()), "same dtype"), (dict(k=x.double(), v=x.double()), "dtype"),
                    (dict(v=x[:, :, :2]), "shape"), (dict(k=x.transpose(2, 3)), "shape"),
                    (dict(k=torch.zeros(2, 3, 64, 64, dtype=torch.bfloat16).transpose(2, 3),
                          v=torch.zeros(2, 3, 64, 64, dtype=torch.bfloat16)), "contiguous"),
                    (dict(counts=ints.float()), "float32"), (dict(k=x[:, :, :0], v=x[:, :, :0]), "at least 1")]:
        a = {**good, **kw}
        with pytest.raises(ValueError, match=msg):
            vq.vq_paged_append(desc, cache, a.pop("block_table"), a.pop("start"), a.pop("k"), a.pop("v"), **a)
    q = torch.zeros(2, 6, 4, 64, dtype=torch.bfloat16)
    for kw, msg in [(dict(q=q.float()), "dtype"), (dict(out=q.half()), "same dtype"), (dict(out=q[:, :3]), "shape"),
                    (dict(lse=torch.zeros(2, 6, 3)), "shape"), (dict(slopes=torch.zeros(3)), "shape"),
                    (dict(slopes=torch.zeros(6, dtype=torch.float64)), "float64"),
                    (dict(first=torch.zeros(2, 5, dtype=torch.int32)), "shape"), (dict(q_lens=ints.long()), "int64")]:
        a = {**dict(q=q, out=q), **kw}
        with pytest.raises(ValueError, match=msg):
            vq.vq_paged_attention(desc, cache, table, ints, a.pop("q"), 0.1, a.pop("out"), **a)
    bare = vq.PagedCache(desc, device="cpu")
    with pytest.raises(ValueError, match="weight"):
        vq.vq_paged_weights(desc, bare, table, ints, q, 0.1, torch.zeros(2, 6, 4))
    kept = torch.zeros(2, 3, 8, dtype=torch.int32)
    with pytest.raises(ValueError, match="weight"):
        vq.vq_paged_evict(desc, bare, table, ints, desc, cache, table, ints, 8, kept=kept)
    with pytest.raises(ValueError, match="kept"):
        vq.vq_paged_evict(desc, cache, table, ints, desc, cache, table, ints, 9, kept=kept)


def test_launch_without_gpu_reports_cuda_error():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _append() == vq.VQ_ERR_CUDA and _evict() == vq.VQ_ERR_CUDA and _attention() == vq.VQ_ERR_CUDA


def test_packed_query_is_the_c_structure():
    fields = [2, 6, 4, 2, 0x10, 1, 2, 3, 0x20, 0x30, 0x40, 0x50, 0x60, 0x70, 0x80, 0.5, 30.0, 1]
    raw = vq._QUERY.pack(*fields)
    q = vq.vq_paged_query.from_buffer_copy(raw.ljust(ctypes.sizeof(vq.vq_paged_query), b"\0"))
    got = []
    for name, _ in vq.vq_paged_query._fields_:
        v = getattr(q, name)
        got += list(v) if name == "q_strides" else [v]
    assert got == fields and ctypes.sizeof(vq.vq_paged_query) - len(raw) in (0, 4)
