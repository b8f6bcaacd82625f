// Eviction from the paged cache: per (sequence, head) the tokens of largest
// accumulated attention weight are kept, with the first `sinks` and the last
// `recent` ones, and moved in order into other pages.
//
// Which tokens: of the len - sinks - recent that are not safe, the `keep - sinks -
// recent` largest weights; equal weights go to the lowest slot, a NaN counts as minus
// infinity. Order is that of the weights' bits as unsigned keys (sign folded, -0 as
// +0), and the cut is found digit by digit from the top: the largest key T such that
// at least as many keys as wanted are >= T.
//
// The move keeps codes wherever it can: a page's scale is the largest of its tokens'
// old scales, so tokens from a page of that scale keep their codes to the bit, and
// others are rounded once, code * (old / new). (Scales from the kept tokens' own maximum
// would fit tighter but re-round every code.)
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "paged.cuh"
#include "vq_internal.h"

namespace vq {

struct PagedEvictParams {
  PagedPool from, to;
  const int32_t* lens;
  int32_t* to_lens;
  int32_t* kept;  // [B][H][keep]
  int B, keep, sinks, recent;
};

namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectBins = 2048;         // digits of 11, 11 and 10 bits
constexpr int kSelectCached = 48 * 1024;  // keys that shared memory holds; later ones are read again for each digit

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0x007fffffu;  // as minus infinity
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum of one number per thread over the CTA, and the total. `sums`: one word per warp.
__device__ __forceinline__ int block_scan(int x, int* sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) sums[warp] = y;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSelectThreads / 32; ++w) {
    const int s = sums[w];
    before += w < warp ? s : 0;
    total += s;
  }
  __syncthreads();
  return before + y - x;
}

// One CTA per (sequence, head). Its keys are gathered once into shared memory (a slot's page is looked up, then its
// weight: kept there, the digits cost no global memory); three passes for the digits of the cut, one to write the kept
// slots in order. Counts are whole numbers: their order does not matter.
__global__ void __launch_bounds__(kSelectThreads) paged_select_kernel(const __grid_constant__ PagedEvictParams p, int cached) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem_raw);
  __shared__ int hist[kSelectBins];
  __shared__ int sums[kSelectThreads / 32];
  __shared__ uint32_t sm_prefix;
  __shared__ int sm_want;
  const int b = blockIdx.x / p.from.H, h = blockIdx.x % p.from.H;
  const int tid = threadIdx.x;
  const int len = paged_len(p.from, p.lens, b);
  int32_t* kept = p.kept + static_cast<int64_t>(blockIdx.x) * p.keep;
  const int held = min(len, p.keep);
  for (int i = tid + held; i < p.keep; i += kSelectThreads) kept[i] = -1;
  if (h == 0 && tid == 0) p.to_lens[b] = held;
  if (len <= p.keep) {
    for (int i = tid; i < held; i += kSelectThreads) kept[i] = i;
    return;
  }
  const int lo = p.sinks, hi = len - p.recent;  // the slots that compete
  const int want = p.keep - p.sinks - p.recent;
  auto gather = [&](int slot) -> uint32_t {
    const int page = paged_page(p.from, b, slot / kPage);
    if (page < 0) return 0x007fffffu;
    return weight_key(__ldg(p.from.weight + (static_cast<int64_t>(page) * p.from.H + h) * kPage + slot % kPage));
  };
  auto key = [&](int slot) -> uint32_t { return slot < cached ? keys[slot] : gather(slot); };
  const int there = min(len, cached);
#pragma unroll 8
  for (int s = tid; s < there; s += kSelectThreads) keys[s] = gather(s);
  uint32_t prefix = 0;
  int need = want;
  if (want > 0) {
#pragma unroll 1
    for (int digit = 0; digit < 3; ++digit) {
      const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
      const uint32_t bins = digit == 2 ? 1023u : 2047u;
      const uint32_t mask = digit == 0 ? 0u : ~0u << (digit == 1 ? 21 : 10);
      hist[tid] = hist[tid + kSelectThreads] = 0;
      __syncthreads();
      for (int s = lo + tid; s < hi; s += kSelectThreads) {
        const uint32_t k = key(s);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & bins], 1);
      }
      __syncthreads();
      // the highest digit with at least `need` keys at it or above: two bins per thread, from the top
      const int top = kSelectBins - 1 - 2 * tid;
      const int c0 = hist[top], c1 = hist[top - 1];
      int all;
      const int before = block_scan(c0 + c1, sums, all);
      if (before < need && before + c0 + c1 >= need) {
        const bool second = before + c0 < need;
        sm_prefix = prefix | (static_cast<uint32_t>(top - second) << shift);
        sm_want = need - before - (second ? c0 : 0);
      }
      __syncthreads();
      prefix = sm_prefix;
      need = sm_want;
    }
  } else {
    __syncthreads();
  }
  // prefix: the cut; `need` of the keys equal to it are kept, the lowest slots
  int done = 0, ties = 0;  // kept slots and ties before this tile of slots
#pragma unroll 1
  for (int s0 = 0; s0 < len; s0 += kSelectThreads) {
    const int s = s0 + tid;
    bool in = false, tie = false;
    if (s < len) {
      in = s < lo || s >= hi;
      if (!in && want > 0) {
        const uint32_t k = key(s);
        in = k > prefix;
        tie = k == prefix;
      }
    }
    // both counts in one sum: at most 1024 of each
    int all;
    const int before = block_scan((in ? 1 : 0) | (tie ? 1 << 16 : 0), sums, all);
    const int tie_before = ties + (before >> 16);
    // ties before this slot that are kept take a place each
    const int place = done + (before & 0xffff) + min(tie_before, need);
    if ((in || (tie && tie_before < need)) && place < held) kept[place] = s;
    done += all & 0xffff;
    ties += all >> 16;
  }
}

// Two e4m3 codes times a power of two, rounded again.
__device__ __forceinline__ uint32_t e4m3_scaled(uint32_t pair, __half2 g) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(pair)));
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h2), g);
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&v)));
  return r;
}

// One CTA per (destination page, head, sequence): gathers its tokens' codes. Bound by memory (with the selection, 8 x 12
// heads of 18720 tokens down to 9360: 130 us, 3.6 TB/s).
template <int CODE, int D>
__global__ void __launch_bounds__(128) paged_move_kernel(const __grid_constant__ PagedEvictParams p) {
  constexpr int LPR = D / 16, RPI = 128 / LPR;
  __shared__ int64_t sm_src[kPage];  // (page * H + head) * 64 + slot, -1: none
  __shared__ float sm_scale[2][kPage];
  __shared__ float sm_ratio[2][kPage];  // old scale over the page's new one
  __shared__ float sm_top[2];            // the new one
  const int per = (p.keep + kPage - 1) / kPage;
  const int tile = blockIdx.x % per, bh = blockIdx.x / per;
  const int b = bh / p.from.H, h = bh - b * p.from.H;
  const int tid = threadIdx.x;
  const int held = min(paged_len(p.from, p.lens, b), p.keep) - tile * kPage;  // tokens of this page
  if (held <= 0) return;
  const int page = paged_page(p.to, b, tile);
  if (page < 0) return;
  const int64_t dst = static_cast<int64_t>(page) * p.to.H + h;
  if (tid < kPage) {
    int64_t src = -1;
    float s0 = 0.0f, s1 = 0.0f;
    if (tid < held) {
      const int slot = __ldg(p.kept + static_cast<int64_t>(bh) * p.keep + tile * kPage + tid);
      const int from = slot >= 0 ? paged_page(p.from, b, slot / kPage) : -1;
      if (from >= 0) {
        const int64_t ph = static_cast<int64_t>(from) * p.from.H + h;
        src = ph * kPage + slot % kPage;
        s0 = __ldg(p.from.scale[0] + ph);
        s1 = __ldg(p.from.scale[1] + ph);
      }
      if (p.to.weight) p.to.weight[dst * kPage + tid] = src >= 0 ? __ldg(p.from.weight + src) : 0.0f;
      if (p.to.pos) p.to.pos[dst * kPage + tid] = src >= 0 && p.from.pos ? __ldg(p.from.pos + src) : slot;
    }
    sm_src[tid] = src;
    sm_scale[0][tid] = s0;
    sm_scale[1][tid] = s1;
  }
  __syncthreads();
  {  // two warps per tensor
    const int t = tid >> 6;
    float top = fmaxf(sm_scale[t][tid & 31], sm_scale[t][32 + (tid & 31)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 63) == 0) p.to.scale[t][dst] = sm_top[t] = top;
    const float s = sm_scale[t][tid & 63];
    sm_ratio[t][tid & 63] = s == top ? 1.0f : __fdiv_rn(s, top);
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int c = (tid % LPR) * 16;
    uint4 v[kPage / RPI];
#pragma unroll
    for (int i = 0; i < kPage / RPI; ++i) {
      const int64_t src = sm_src[i * RPI + tid / LPR];
      v[i] = src >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.from.code[t] + src * D + c)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kPage / RPI; ++i) {
      const int slot = i * RPI + tid / LPR;
      if (slot >= held) continue;
      const float ratio = sm_ratio[t][slot];
      if (sm_scale[t][slot] != sm_top[t]) {
        if (CODE == kCodeInt8) {
          // the quotient code * old / new in float32 is off by less than 127 * 2^-22; next to a half it is taken in 64
          // bits, where code * old is exact and the quotient either a half exactly or at least 2^-33 from one: it
          // rounds as the real number does (a ratio rounded first would miss the halves)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t o = (&v[i].x)[w];
            uint32_t r = 0;
            bool near = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float q = code_value<CODE>((o >> (8 * j)) & 0xff) * ratio;
              const int k = __float2int_rn(q);
              near |= fabsf(q - static_cast<float>(k)) > 0.4999f;
              r |= (static_cast<uint32_t>(k) & 0xff) << (8 * j);
            }
            if (near) {
              const double from = sm_scale[t][slot], to = sm_top[t];
              r = 0;
#pragma unroll 1
              for (int j = 0; j < 4; ++j) {
                const int k = __double2int_rn(static_cast<double>(code_value<CODE>((o >> (8 * j)) & 0xff)) * from / to);
                r |= (static_cast<uint32_t>(k) & 0xff) << (8 * j);
              }
            }
            (&v[i].x)[w] = r;
          }
        } else {
          // a power of two (2^-24 and less leave nothing of any code): exact in fp16 wherever the result is not 0
          const __half2 g = __half2half2(__float2half_rn(ratio));
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t o = (&v[i].x)[w];
            (&v[i].x)[w] = e4m3_scaled(o & 0xffffu, g) | (e4m3_scaled(o >> 16, g) << 16);
          }
        }
      }
      *reinterpret_cast<uint4*>(p.to.code[t] + (dst * kPage + slot) * D + c) = v[i];
    }
  }
}

}  // namespace

inline cudaError_t launch_paged_evict(const PagedEvictParams& p, int code, cudaStream_t stream) {
  static bool configured[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(paged_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectCached * 4);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const unsigned heads = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.from.H);
  const int64_t slots = static_cast<int64_t>(p.from.max_pages) * kPage;
  const int cached = static_cast<int>(slots < kSelectCached ? slots : kSelectCached);
  paged_select_kernel<<<heads, kSelectThreads, cached * 4, stream>>>(p, cached);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned grid = heads * static_cast<unsigned>((p.keep + kPage - 1) / kPage);
  if (code == kCodeInt8) {
    if (p.from.D == 64)
      paged_move_kernel<kCodeInt8, 64><<<grid, 128, 0, stream>>>(p);
    else
      paged_move_kernel<kCodeInt8, 128><<<grid, 128, 0, stream>>>(p);
  } else {
    if (p.from.D == 64)
      paged_move_kernel<kCodeE4m3, 64><<<grid, 128, 0, stream>>>(p);
    else
      paged_move_kernel<kCodeE4m3, 128><<<grid, 128, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace vq
