// Which kernel a call on the paged cache takes, how it is split, and its launch.
#pragma once

#include "paged_attention.cuh"
#include "paged_many.cuh"
#include "paged_weights.cuh"

namespace vq {

// rows to a tile: 8 or 16 (paged_few_kernel, of `warps` warps) or 256 (paged_many_kernel).
struct PagedPlan {
  int rows, row_tiles, splits, warps;
};

// Up to so many pages a CTA of 12 warps takes a sequence whole where CTAs are few: no join after it (16 heads of 680
// tokens: 7.0 against 9.0 us with two splits of 4 warps and a join).
constexpr int kAlonePages = 32;
// At most so many rows per key head take the few-row kernels, which read the codes once per 8 or 16 rows; above, the
// tensor cores' tiles of 256 rows win. Few-row against many-row kernel, 8192 tokens, head_dim 128, int8: 8 sequences of
// 8 heads, 32 rows 92 against 125 us, 48 rows 127 against 127, 64 rows 152 against 127; one sequence, 48 rows 35 against
// 31 us; 32 sequences, 48 rows 371 against 440 us, 64 rows 471 against 436. The weights at 48 rows: 86 against 121, 29
// against 22, 229 against 440 us.
constexpr int kFewRows = 48;

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
    // Four CTAs per SM, while a split has two pages for each of its four warps; where a split then still has 16 pages,
    // up to four times as many, so that sequences of different lengths even out (32 ragged sequences of 8 heads: 107 us
    // with 3 splits, 100 with 10). Short sequences that make three CTAs per SM as they are stay whole (512 of up to 2000
    // tokens: 47 us against 53 with 2).
    want = (4 * static_cast<int64_t>(sms) + base - 1) / base;
    most = (max_pages + 7) / 8;
    const int64_t even = (16 * static_cast<int64_t>(sms) + base - 1) / base, long_ones = max_pages / 16;
    want = want < most ? want : most;
    most = even < long_ones ? even : long_ones;
    want = most = want > most ? want : most;
    if (base >= 3 * static_cast<int64_t>(sms) && max_pages <= 2 * kAlonePages) want = 1;
  }
  const int64_t s = want < most ? want : most;
  plan.splits = static_cast<int>(s > 1 ? s : 1);
  plan.warps = kFewWarps;
  if (plan.rows == 8 && base < 2 * static_cast<int64_t>(sms) && max_pages <= kAlonePages) {
    plan.splits = 1;
    plan.warps = kFewWarpsAlone;
  }
  return plan;
}

// Partial outputs and their references and sums, one row per split.
inline size_t paged_plan_bytes(const PagedPlan& plan, int B, int H, int D) {
  if (plan.splits <= 1) return 0;
  const size_t rows = static_cast<size_t>(plan.splits) * B * H * plan.row_tiles * plan.rows;
  return rows * (static_cast<size_t>(D) * 4 + 8);
}

namespace {

// Launches Kernel with `smem` bytes of dynamic shared memory, allowed once per device.
template <auto Kernel>
cudaError_t launch_paged(const PagedAttnParams& p, unsigned grid, int threads, int smem, cudaStream_t stream) {
  static bool configured[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  Kernel<<<grid, threads, smem, stream>>>(p);
  return cudaGetLastError();
}

// f(head_dim tag, code tag, mode tag) for the call's variant.
template <typename F>
cudaError_t paged_variant(const PagedAttnParams& p, int code, F f) {
  const bool general = p.slopes || (p.c.pos && (p.first || (p.prefix && p.causal)));
  auto by_mode = [&](auto d, auto c) {
    if (general) return f(d, c, std::integral_constant<int, kGeneral>{});
    if (p.cap > 0.0f) return f(d, c, std::integral_constant<int, kCap>{});
    return f(d, c, std::integral_constant<int, kPlain>{});
  };
  auto by_code = [&](auto d) {
    return code == kCodeInt8 ? by_mode(d, std::integral_constant<int, kCodeInt8>{})
                             : by_mode(d, std::integral_constant<int, kCodeE4m3>{});
  };
  return p.c.D == 64 ? by_code(std::integral_constant<int, 64>{}) : by_code(std::integral_constant<int, 128>{});
}

}  // namespace

inline cudaError_t launch_paged_attention(PagedAttnParams& p, const PagedPlan& plan, int code, void* workspace,
                                          cudaStream_t stream) {
  p.row_tiles = plan.row_tiles;
  p.splits = plan.splits;
  const size_t rows = static_cast<size_t>(plan.splits) * p.B * p.c.H * plan.row_tiles * plan.rows;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + rows * p.c.D);
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.c.H * plan.row_tiles * plan.splits);
  cudaError_t e = paged_variant(p, code, [&](auto d, auto c, auto m) {
    constexpr int D = decltype(d)::value, CODE = decltype(c)::value, MODE = decltype(m)::value;
    constexpr int W = kFewWarps, A = kFewWarpsAlone;
    if (plan.rows == 8 && plan.warps == A)
      return launch_paged<paged_few_kernel<D, CODE, 8, MODE, A>>(p, grid, A * 32, FewCfg<D, 8, A>::SMEM, stream);
    if (plan.rows == 8)
      return launch_paged<paged_few_kernel<D, CODE, 8, MODE, W>>(p, grid, W * 32, FewCfg<D, 8, W>::SMEM, stream);
    if (plan.rows == 16)
      return launch_paged<paged_few_kernel<D, CODE, 16, MODE, W>>(p, grid, W * 32, FewCfg<D, 16, W>::SMEM, stream);
    return launch_paged<paged_many_kernel<D, CODE, MODE>>(p, grid, ManyCfg<D>::THREADS, ManyCfg<D>::SMEM_ALLOC, stream);
  });
  if (e != cudaSuccess || plan.splits <= 1) return e;
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.Hq * p.n);
  const int pad = plan.row_tiles * plan.rows;
  if (p.c.D == 64)
    plan.splits > 32 ? paged_join_kernel<64, 16><<<blocks, 512, 0, stream>>>(p, pad)
                     : paged_join_kernel<64, 4><<<blocks, 128, 0, stream>>>(p, pad);
  else
    plan.splits > 32 ? paged_join_kernel<128, 16><<<blocks, 512, 0, stream>>>(p, pad)
                     : paged_join_kernel<128, 4><<<blocks, 128, 0, stream>>>(p, pad);
  return cudaGetLastError();
}

inline cudaError_t launch_paged_weights(PagedAttnParams& p, int code, int sms, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.n) * p.G;
  return paged_variant(p, code, [&](auto d, auto c, auto m) {
    constexpr int D = decltype(d)::value, CODE = decltype(c)::value, MODE = decltype(m)::value;
    if (rows > kFewRows) {
      const int64_t grid = static_cast<int64_t>(p.B) * p.c.H * ((p.c.max_pages + 1) / 2);
      return launch_paged<paged_sums_kernel<D, CODE, MODE>>(p, static_cast<unsigned>(grid), SumCfg<D>::THREADS,
                                                            SumCfg<D>::SMEM_ALLOC, stream);
    }
    p.splits = paged_plan(p.B, p.c.H, 16, 1, p.c.max_pages, sms).splits;  // (one tile of rows: split as its attention is)
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.c.H * p.splits);
    if (rows <= 8)
      return launch_paged<paged_weights_kernel<D, CODE, 8, MODE>>(p, grid, kFewWarps * 32, kFewWarps * kSumStages * UnitCfg<D>::K, stream);
    return launch_paged<paged_weights_kernel<D, CODE, 16, MODE>>(p, grid, kFewWarps * 32, kFewWarps * kSumStages * UnitCfg<D>::K, stream);
  });
}

}  // namespace vq
