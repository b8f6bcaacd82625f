// Which kernel a call on the paged cache takes, how it is split, and its launch.
#pragma once

#include "paged_attention.cuh"
#include "paged_many.cuh"
#include "paged_weights.cuh"

namespace vq {

// rows to a tile: 8 or 16 (paged_few_kernel) or 256 (paged_many_kernel).
struct PagedPlan {
  int rows, row_tiles, splits;
};

constexpr int kFewRows = 32;  // at most so many rows per key head take the few-row kernel

inline PagedPlan paged_plan(int B, int H, int G, int n, int max_pages, int sms) {
  PagedPlan plan;
  const int64_t rows = static_cast<int64_t>(G) * n;
  plan.rows = rows <= 8 ? 8 : rows <= kFewRows ? 16 : 256;
  plan.row_tiles = static_cast<int>((rows + plan.rows - 1) / plan.rows);
  const int64_t base = static_cast<int64_t>(B) * H * plan.row_tiles;
  int64_t want, most;
  if (plan.rows == 256) {
    // one CTA per SM; a split has at least four tiles of two pages
    want = sms / base;
    most = max_pages / 8;
  } else {
    // about three CTAs per SM; a split has two pages for each of its four warps
    want = (3 * static_cast<int64_t>(sms) + base - 1) / base;
    most = (max_pages + 7) / 8;
  }
  const int64_t s = want < most ? want : most;
  plan.splits = static_cast<int>(s > 1 ? s : 1);
  return plan;
}

// Partial outputs and their references and sums, one row per split.
inline size_t paged_plan_bytes(const PagedPlan& plan, int B, int H, int D) {
  if (plan.splits <= 1) return 0;
  const size_t rows = static_cast<size_t>(plan.splits) * B * H * plan.row_tiles * plan.rows;
  return rows * (static_cast<size_t>(D) * 4 + 8);
}

inline bool paged_biased(const PagedAttnParams& p) {
  return p.cap > 0.0f || p.slopes || p.first || (p.prefix && p.causal);
}

inline cudaError_t launch_paged_attention(PagedAttnParams& p, const PagedPlan& plan, int code, void* workspace,
                                          cudaStream_t stream) {
  p.row_tiles = plan.row_tiles;
  p.splits = plan.splits;
  const size_t rows = static_cast<size_t>(plan.splits) * p.B * p.c.H * plan.row_tiles * plan.rows;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + rows * p.c.D);
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.c.H * plan.row_tiles * plan.splits);
  cudaError_t e = plan.rows == 256 ? launch_paged_many(p, code, grid, stream) :
                                   paged_attn_dispatch(p.c.D, code, paged_biased(p), [&](auto d, auto c, auto bias) {
    if (plan.rows == 8)
      paged_few_kernel<d(), c(), 8, bias()><<<grid, kFewWarps * 32, 0, stream>>>(p);
    else
      paged_few_kernel<d(), c(), 16, bias()><<<grid, kFewWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
  });
  if (e != cudaSuccess || plan.splits <= 1) return e;
  const int64_t warps = static_cast<int64_t>(p.B) * p.c.H * p.n * p.G;
  const unsigned blocks = static_cast<unsigned>((warps + 3) / 4);
  if (p.c.D == 64)
    paged_join_kernel<64><<<blocks, 128, 0, stream>>>(p, plan.row_tiles * plan.rows);
  else
    paged_join_kernel<128><<<blocks, 128, 0, stream>>>(p, plan.row_tiles * plan.rows);
  return cudaGetLastError();
}

inline cudaError_t launch_paged_weights(PagedAttnParams& p, int code, cudaStream_t stream) {
  const int64_t grid = static_cast<int64_t>(p.B) * p.c.H * ((p.c.max_pages + 1) / 2);
  if (static_cast<int64_t>(p.n) * p.G > kFewRows)
    return many_dispatch(p, code, [&](auto d, auto c, auto m) {
      return launch_sums_variant<d(), c(), m()>(p, static_cast<unsigned>(grid), stream);
    });
  return paged_attn_dispatch(p.c.D, code, paged_biased(p), [&](auto d, auto c, auto bias) {
    paged_weights_kernel<d(), c(), bias()><<<static_cast<unsigned>(grid), kFewWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
  });
}

}  // namespace vq
