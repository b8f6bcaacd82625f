// C ABI of the paged 8-bit cache: argument validation and launches (see
// include/vq.h for the contract of each call). Part of the library's one
// translation unit, after the block cache's entry points, whose error helpers it
// uses.
#pragma once

#include "paged.cuh"
#include "paged_evict.cuh"
#include "paged_launch.cuh"

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

vq_status check_paged_desc(const vq_paged_desc* d) {
  if (!d) return fail(VQ_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->kv_heads < 1 || d->num_pages < 1 || d->max_pages < 1)
    return fail(VQ_ERR_INVALID_ARGUMENT, "kv_heads, num_pages and max_pages must be >= 1");
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(VQ_ERR_UNSUPPORTED, "head_dim %d unsupported (64 or 128)", d->head_dim);
  if (d->code != VQ_INT8 && d->code != VQ_E4M3) return fail(VQ_ERR_UNSUPPORTED, "code %d unsupported", d->code);
  if (d->max_pages > (1 << 24)) return fail(VQ_ERR_UNSUPPORTED, "max_pages %d too large (2^24)", d->max_pages);
  if (int64_t(d->num_pages) * d->kv_heads > (int64_t(1) << 31))
    return fail(VQ_ERR_UNSUPPORTED, "pool of %d pages x %d heads too large", d->num_pages, d->kv_heads);
  return VQ_OK;
}

vq_status check_paged_cache(const vq_paged_cache* c) {
  if (!c) return fail(VQ_ERR_INVALID_ARGUMENT, "cache is NULL");
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return fail(VQ_ERR_INVALID_ARGUMENT, "cache has a NULL pointer");
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale) || !aligned16(c->pos) ||
      !aligned16(c->weight))
    return fail(VQ_ERR_MISALIGNED, "cache pointers must be 16-byte aligned");
  return VQ_OK;
}

vq_status check_table(const int32_t* table, const int32_t* lens, const char* lens_name) {
  if (!table || !lens) return fail(VQ_ERR_INVALID_ARGUMENT, "block_table or %s is NULL", lens_name);
  if (!aligned4(table) || !aligned4(lens)) return fail(VQ_ERR_MISALIGNED, "block_table or %s is not 4-byte aligned", lens_name);
  return VQ_OK;
}

// Strides of a tensor that is written: no two elements at one address by a zero stride.
vq_status check_out_strides(const int64_t st[3], int esize, const int64_t extent[3], const char* name) {
  vq_status s = check_strides(st, esize, name);
  if (s != VQ_OK) return s;
  for (int i = 0; i < 3; ++i)
    if (st[i] == 0 && extent[i] > 1) return fail(VQ_ERR_INVALID_ARGUMENT, "%s stride %d is 0", name, i);
  return VQ_OK;
}

vq_status check_grid(int64_t blocks) {
  if (blocks > INT32_MAX) return fail(VQ_ERR_UNSUPPORTED, "call too large: %lld blocks", (long long)blocks);
  return VQ_OK;
}

vq::PagedPool paged_pool(const vq_paged_desc* d, const vq_paged_cache* c, const int32_t* table) {
  vq::PagedPool p{};
  p.code[0] = static_cast<unsigned char*>(c->k);
  p.code[1] = static_cast<unsigned char*>(c->v);
  p.scale[0] = c->k_scale;
  p.scale[1] = c->v_scale;
  p.pos = c->pos;
  p.weight = c->weight;
  p.table = table;
  p.H = d->kv_heads;
  p.D = d->head_dim;
  p.num_pages = d->num_pages;
  p.max_pages = d->max_pages;
  return p;
}

// Streaming multiprocessors of the current device, asked for once per device.
cudaError_t paged_sms(int* sms) {
  static int known[vq::kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= vq::kMaxDevices) return cudaErrorInvalidDevice;
  if (!known[dev]) {
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    known[dev] = n;
  }
  *sms = known[dev];
  return cudaSuccess;
}

vq_status check_heads(const vq_paged_desc* d, int32_t batch, int32_t q_heads, int32_t n) {
  if (batch < 1 || n < 1 || q_heads < 1) return fail(VQ_ERR_INVALID_ARGUMENT, "batch, q_heads and n must be >= 1");
  if (q_heads % d->kv_heads != 0)
    return fail(VQ_ERR_INVALID_ARGUMENT, "q_heads %d is not a multiple of kv_heads %d", q_heads, d->kv_heads);
  if (int64_t(q_heads) * n > (int64_t(1) << 30)) return fail(VQ_ERR_UNSUPPORTED, "call too large: %d queries", n);
  return VQ_OK;
}

// The checks that attention and weights share; fills the kernels' parameters.
vq_status build_paged_query(const vq_paged_desc* desc, const vq_paged_cache* cache, const vq_paged_query* q,
                            vq::PagedAttnParams& p) {
  vq_status st = check_paged_desc(desc);
  if (st != VQ_OK) return st;
  if ((st = check_paged_cache(cache)) != VQ_OK) return st;
  if (!q || !q->q) return fail(VQ_ERR_INVALID_ARGUMENT, "query or q is NULL");
  if ((st = check_heads(desc, q->batch, q->q_heads, q->n)) != VQ_OK) return st;
  if (q->dtype != VQ_BF16 && q->dtype != VQ_F16) return fail(VQ_ERR_UNSUPPORTED, "query dtype %d unsupported", int(q->dtype));
  if (!aligned16(q->q)) return fail(VQ_ERR_MISALIGNED, "q must be 16-byte aligned");
  if ((st = check_strides(q->q_strides, 2, "q")) != VQ_OK) return st;
  if ((st = check_table(q->block_table, q->lens, "lens")) != VQ_OK) return st;
  if (!aligned4(q->q_lens) || !aligned4(q->q_pos) || !aligned4(q->prefix) || !aligned4(q->first) || !aligned4(q->slopes))
    return fail(VQ_ERR_MISALIGNED, "q_lens, q_pos, prefix, first and slopes must be 4-byte aligned");
  if (!(q->softmax_scale > 0.0f) || q->softmax_scale > 1e6f)
    return fail(VQ_ERR_INVALID_ARGUMENT, "softmax_scale must be in (0, 1e6]");
  if (!(q->softcap >= 0.0f) || q->softcap > 1e6f) return fail(VQ_ERR_INVALID_ARGUMENT, "softcap must be in [0, 1e6]");
  if (q->softcap > 0.0f && q->softcap < 1e-6f) return fail(VQ_ERR_INVALID_ARGUMENT, "softcap must be 0 or at least 1e-6");
  if (q->causal != 0 && q->causal != 1) return fail(VQ_ERR_INVALID_ARGUMENT, "causal must be 0 or 1");
  if (q->prefix && !q->causal) return fail(VQ_ERR_INVALID_ARGUMENT, "prefix without causal: every token is seen already");
  p = vq::PagedAttnParams{};
  p.c = paged_pool(desc, cache, q->block_table);
  p.lens = q->lens;
  p.q_lens = q->q_lens;
  p.q_pos = q->q_pos;
  p.prefix = q->prefix;
  p.first = q->first;
  p.slopes = q->slopes;
  p.q = static_cast<const uint16_t*>(q->q);
  p.q_sb = q->q_strides[0];
  p.q_sh = q->q_strides[1];
  p.q_st = q->q_strides[2];
  p.B = q->batch;
  p.Hq = q->q_heads;
  p.G = q->q_heads / desc->kv_heads;
  p.n = q->n;
  p.causal = q->causal;
  p.q_bf16 = q->dtype == VQ_BF16;
  p.sigma = q->softmax_scale;
  p.cap = q->softcap;
  return VQ_OK;
}

}  // namespace

extern "C" {

vq_status vq_paged_append(const vq_paged_desc* desc, const vq_paged_cache* cache, int32_t batch, int32_t n,
                          const void* k, const void* v, vq_dtype dtype, const int64_t k_strides[3],
                          const int64_t v_strides[3], const int32_t* block_table, const int32_t* start,
                          const int32_t* counts, const int32_t* pos, void* stream) {
  vq_status st = check_paged_desc(desc);
  if (st != VQ_OK) return st;
  if ((st = check_paged_cache(cache)) != VQ_OK) return st;
  if (batch < 1 || n < 1) return fail(VQ_ERR_INVALID_ARGUMENT, "batch and n must be >= 1");
  if (dtype != VQ_BF16 && dtype != VQ_F32 && dtype != VQ_F16) return fail(VQ_ERR_UNSUPPORTED, "dtype %d unsupported", int(dtype));
  if (!k || !v) return fail(VQ_ERR_INVALID_ARGUMENT, "k or v is NULL");
  if (!aligned16(k) || !aligned16(v)) return fail(VQ_ERR_MISALIGNED, "k and v must be 16-byte aligned");
  const int esize = dtype == VQ_F32 ? 4 : 2;
  if ((st = check_strides(k_strides, esize, "k")) != VQ_OK) return st;
  if ((st = check_strides(v_strides, esize, "v")) != VQ_OK) return st;
  if ((st = check_table(block_table, start, "start")) != VQ_OK) return st;
  if (!aligned4(counts) || !aligned4(pos)) return fail(VQ_ERR_MISALIGNED, "counts and pos must be 4-byte aligned");
  vq::PagedAppendParams p{};
  p.c = paged_pool(desc, cache, block_table);
  p.x[0] = k;
  p.x[1] = v;
  for (int t = 0; t < 2; ++t) {
    const int64_t* s = t ? v_strides : k_strides;
    p.sb[t] = s[0];
    p.sh[t] = s[1];
    p.st[t] = s[2];
  }
  p.start = start;
  p.counts = counts;
  p.pos = pos;
  p.B = batch;
  p.n = n;
  p.tiles = static_cast<int>((int64_t(n) + vq::kPage - 2) / vq::kPage) + 1;
  if ((st = check_grid(int64_t(batch) * desc->kv_heads * p.tiles * 2)) != VQ_OK) return st;
  cudaError_t e = vq::launch_paged_append(p, dtype, desc->code, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged append launch");
  return ok();
}

vq_status vq_paged_read(const vq_paged_desc* desc, const vq_paged_cache* cache, int32_t batch, int32_t n,
                        const int32_t* block_table, const int32_t* start, const int32_t* counts, void* k_out,
                        void* v_out, vq_dtype dtype, const int64_t k_strides[3], const int64_t v_strides[3],
                        void* stream) {
  vq_status st = check_paged_desc(desc);
  if (st != VQ_OK) return st;
  if ((st = check_paged_cache(cache)) != VQ_OK) return st;
  if (batch < 1 || n < 1) return fail(VQ_ERR_INVALID_ARGUMENT, "batch and n must be >= 1");
  if (dtype != VQ_BF16 && dtype != VQ_F32 && dtype != VQ_F16) return fail(VQ_ERR_UNSUPPORTED, "dtype %d unsupported", int(dtype));
  if (!k_out || !v_out) return fail(VQ_ERR_INVALID_ARGUMENT, "k_out or v_out is NULL");
  if (!aligned16(k_out) || !aligned16(v_out)) return fail(VQ_ERR_MISALIGNED, "k_out and v_out must be 16-byte aligned");
  const int esize = dtype == VQ_F32 ? 4 : 2;
  const int64_t extent[3] = {batch, desc->kv_heads, n};
  if ((st = check_out_strides(k_strides, esize, extent, "k_out")) != VQ_OK) return st;
  if ((st = check_out_strides(v_strides, esize, extent, "v_out")) != VQ_OK) return st;
  if ((st = check_table(block_table, start, "start")) != VQ_OK) return st;
  if (!aligned4(counts)) return fail(VQ_ERR_MISALIGNED, "counts must be 4-byte aligned");
  vq::PagedReadParams p{};
  p.c = paged_pool(desc, cache, block_table);
  p.out[0] = k_out;
  p.out[1] = v_out;
  for (int t = 0; t < 2; ++t) {
    const int64_t* s = t ? v_strides : k_strides;
    p.sb[t] = s[0];
    p.sh[t] = s[1];
    p.st[t] = s[2];
  }
  p.start = start;
  p.counts = counts;
  p.B = batch;
  p.n = n;
  p.tiles = static_cast<int>((int64_t(n) + vq::kPage - 1) / vq::kPage);
  if ((st = check_grid(int64_t(batch) * desc->kv_heads * p.tiles * 2)) != VQ_OK) return st;
  cudaError_t e = vq::launch_paged_read(p, dtype, desc->code, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged read launch");
  return ok();
}

vq_status vq_paged_attention_workspace(const vq_paged_desc* desc, int32_t batch, int32_t q_heads, int32_t n,
                                       size_t* bytes) {
  vq_status st = check_paged_desc(desc);
  if (st != VQ_OK) return st;
  if ((st = check_heads(desc, batch, q_heads, n)) != VQ_OK) return st;
  if (!bytes) return fail(VQ_ERR_INVALID_ARGUMENT, "bytes is NULL");
  int sms = 0;
  cudaError_t e = paged_sms(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "reading the device's size");
  const vq::PagedPlan plan = vq::paged_plan(batch, desc->kv_heads, q_heads / desc->kv_heads, n, desc->max_pages, sms);
  *bytes = vq::paged_plan_bytes(plan, batch, desc->kv_heads, desc->head_dim);
  return ok();
}

vq_status vq_paged_attention(const vq_paged_desc* desc, const vq_paged_cache* cache, const vq_paged_query* query,
                             void* out, const int64_t out_strides[3], float* lse, void* workspace,
                             size_t workspace_bytes, void* stream) {
  vq::PagedAttnParams p;
  vq_status st = build_paged_query(desc, cache, query, p);
  if (st != VQ_OK) return st;
  if (!out) return fail(VQ_ERR_INVALID_ARGUMENT, "out is NULL");
  if (!aligned16(out) || !aligned16(lse) || !aligned16(workspace))
    return fail(VQ_ERR_MISALIGNED, "out, lse and workspace must be 16-byte aligned");
  const int64_t extent[3] = {p.B, p.Hq, p.n};
  if ((st = check_out_strides(out_strides, 2, extent, "out")) != VQ_OK) return st;
  p.out = static_cast<uint16_t*>(out);
  p.o_sb = out_strides[0];
  p.o_sh = out_strides[1];
  p.o_st = out_strides[2];
  p.lse = lse;
  int sms = 0;
  cudaError_t e = paged_sms(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "reading the device's size");
  const vq::PagedPlan plan = vq::paged_plan(p.B, p.c.H, p.G, p.n, p.c.max_pages, sms);
  const size_t need = vq::paged_plan_bytes(plan, p.B, p.c.H, p.c.D);
  if (need > workspace_bytes || (need && !workspace))
    return fail(VQ_ERR_INVALID_ARGUMENT, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
  if ((st = check_grid(int64_t(p.B) * p.c.H * plan.row_tiles * plan.splits)) != VQ_OK) return st;
  if ((st = check_grid(int64_t(p.B) * p.Hq * p.n)) != VQ_OK) return st;
  e = vq::launch_paged_attention(p, plan, desc->code, workspace, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
  return ok();
}

vq_status vq_paged_weights(const vq_paged_desc* desc, const vq_paged_cache* cache, const vq_paged_query* query,
                           const float* lse, int32_t accumulate, void* stream) {
  vq::PagedAttnParams p;
  vq_status st = build_paged_query(desc, cache, query, p);
  if (st != VQ_OK) return st;
  if (!lse || !cache->weight) return fail(VQ_ERR_INVALID_ARGUMENT, "lse or the cache's weight is NULL");
  if (!aligned16(lse)) return fail(VQ_ERR_MISALIGNED, "lse must be 16-byte aligned");
  if (accumulate != 0 && accumulate != 1) return fail(VQ_ERR_INVALID_ARGUMENT, "accumulate must be 0 or 1");
  p.lse = const_cast<float*>(lse);
  p.accumulate = accumulate;
  if ((st = check_grid(int64_t(p.B) * p.c.H * ((p.c.max_pages + 1) / 2))) != VQ_OK) return st;
  int sms = 0;
  cudaError_t e = paged_sms(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "reading the device's size");
  e = vq::launch_paged_weights(p, desc->code, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged weights launch");
  return ok();
}

vq_status vq_paged_evict(const vq_paged_desc* desc, const vq_paged_cache* cache, int32_t batch,
                         const int32_t* block_table, const int32_t* lens, const vq_paged_desc* to_desc,
                         const vq_paged_cache* to, const int32_t* to_table, int32_t* to_lens, int32_t keep,
                         int32_t sinks, int32_t recent, int32_t* kept, void* stream) {
  vq_status st = check_paged_desc(desc);
  if (st != VQ_OK) return st;
  if ((st = check_paged_desc(to_desc)) != VQ_OK) return st;
  if ((st = check_paged_cache(cache)) != VQ_OK) return st;
  if ((st = check_paged_cache(to)) != VQ_OK) return st;
  if (batch < 1) return fail(VQ_ERR_INVALID_ARGUMENT, "batch must be >= 1");
  if (desc->kv_heads != to_desc->kv_heads || desc->head_dim != to_desc->head_dim || desc->code != to_desc->code)
    return fail(VQ_ERR_INVALID_ARGUMENT, "the two caches differ in kv_heads, head_dim or code");
  if (!cache->weight) return fail(VQ_ERR_INVALID_ARGUMENT, "the cache has no weight");
  if ((st = check_table(block_table, lens, "lens")) != VQ_OK) return st;
  if ((st = check_table(to_table, to_lens, "to_lens")) != VQ_OK) return st;
  if (!kept) return fail(VQ_ERR_INVALID_ARGUMENT, "kept is NULL");
  if (!aligned4(kept)) return fail(VQ_ERR_MISALIGNED, "kept must be 4-byte aligned");
  if (keep < 1 || sinks < 0 || recent < 0 || int64_t(sinks) + recent > keep)
    return fail(VQ_ERR_INVALID_ARGUMENT, "keep %d must be >= 1 and hold sinks %d + recent %d", keep, sinks, recent);
  if ((int64_t(keep) + vq::kPage - 1) / vq::kPage > to_desc->max_pages)
    return fail(VQ_ERR_INVALID_ARGUMENT, "keep %d does not fit the %d pages of a row of to_table", keep, to_desc->max_pages);
  if (lens < to_lens + batch && to_lens < lens + batch)  // heads of a sequence read its length at different times
    return fail(VQ_ERR_INVALID_ARGUMENT, "to_lens overlaps lens");
  vq::PagedEvictParams p{};
  p.from = paged_pool(desc, cache, block_table);
  p.to = paged_pool(to_desc, to, to_table);
  p.lens = lens;
  p.to_lens = to_lens;
  p.kept = kept;
  p.B = batch;
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  if ((st = check_grid(int64_t(batch) * desc->kv_heads * ((int64_t(keep) + vq::kPage - 1) / vq::kPage))) != VQ_OK) return st;
  cudaError_t e = vq::launch_paged_evict(p, desc->code, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged evict launch");
  return ok();
}

}  // extern "C"
