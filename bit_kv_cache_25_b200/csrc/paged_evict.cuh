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

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0x007fffffu;  // as minus infinity
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (sequence, head): four passes over its weights for the digits of the cut
// (8 bits each, counted in shared memory), one to write the kept slots in order.
__global__ void __launch_bounds__(kSelectThreads) paged_select_kernel(const __grid_constant__ PagedEvictParams p) {
  __shared__ int hist[256];
  __shared__ int sm_sum[2][kSelectThreads / 32];
  __shared__ uint32_t sm_prefix;
  __shared__ int sm_want;
  const int b = blockIdx.x / p.from.H, h = blockIdx.x % p.from.H;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = paged_len(p.from, p.lens, b);
  int32_t* kept = p.kept + static_cast<int64_t>(blockIdx.x) * p.keep;
  const int held = min(len, p.keep);
  for (int i = tid + held; i < p.keep; i += kSelectThreads) kept[i] = -1;
  if (h == 0 && tid == 0) p.to_lens[b] = held;
  if (len <= p.keep) {
    for (int i = tid; i < held; i += kSelectThreads) kept[i] = i;
    return;
  }
  const int lo = p.sinks, hi = len - p.recent;  // the tokens that compete
  const int want = p.keep - p.sinks - p.recent;
  auto key = [&](int slot) -> uint32_t {
    const int page = paged_page(p.from, b, slot / kPage);
    if (page < 0) return 0x007fffffu;
    return weight_key(p.from.weight[(static_cast<int64_t>(page) * p.from.H + h) * kPage + slot % kPage]);
  };
  uint32_t prefix = 0;
  int need = want;
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
      for (int s = lo + tid; s < hi; s += kSelectThreads) {
        const uint32_t k = key(s);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 0xff], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // the highest digit d with at least `need` keys at d or above it (8 digits per lane, from the top)
        int own[8], total = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) total += own[j] = hist[255 - (lane * 8 + j)];
        int before = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += y;
        }
        before -= total;
        if (before < need && before + total >= need) {
          int left = need - before, d = 0;
          while (own[d] < left) left -= own[d++];
          sm_prefix = prefix | (static_cast<uint32_t>(255 - (lane * 8 + d)) << shift);
          sm_want = left;
        }
      }
      __syncthreads();
      prefix = sm_prefix;
      need = sm_want;
    }
  }
  // prefix: the cut; `need` of the keys equal to it are kept, the lowest slots
  int done = 0, ties = 0;  // kept slots and ties before this tile of slots
  for (int s0 = 0; s0 < len; s0 += kSelectThreads) {
    const int s = s0 + tid;
    bool safe = false, above = false, tie = false;
    if (s < len) {
      safe = s < lo || s >= hi;
      if (!safe && want > 0) {
        const uint32_t k = key(s);
        above = k > prefix;
        tie = k == prefix;
      }
    }
    const uint32_t tie_mask = __ballot_sync(0xffffffffu, tie), in_mask = __ballot_sync(0xffffffffu, safe || above);
    const uint32_t below = (1u << lane) - 1u;
    if (lane == 0) {
      sm_sum[0][warp] = __popc(in_mask);
      sm_sum[1][warp] = __popc(tie_mask);
    }
    __syncthreads();
    int in_before = done, tie_before = ties, in_all = 0, tie_all = 0;
    for (int w = 0; w < kSelectThreads / 32; ++w) {
      const int a = sm_sum[0][w], t = sm_sum[1][w];
      in_before += w < warp ? a : 0;
      tie_before += w < warp ? t : 0;
      in_all += a;
      tie_all += t;
    }
    in_before += __popc(in_mask & below);
    tie_before += __popc(tie_mask & below);
    // ties before this slot that are kept take a place each
    const int place = in_before + min(tie_before, need);
    if ((safe || above || (tie && tie_before < need)) && place < held) kept[place] = s;
    done += in_all;
    ties += tie_all;
    __syncthreads();
  }
}

// One CTA per (destination page, head, sequence): gathers its tokens' codes.
template <int CODE, int D>
__global__ void __launch_bounds__(128) paged_move_kernel(const __grid_constant__ PagedEvictParams p) {
  constexpr int LPR = D / 16, RPI = 128 / LPR;
  __shared__ int64_t sm_src[kPage];  // (page * H + head) * 64 + slot, -1: none
  __shared__ float sm_scale[2][kPage];
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
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float top = fmaxf(sm_scale[t][tid & 31], sm_scale[t][32 + (tid & 31)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (tid == 0) p.to.scale[t][dst] = top;
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
      const float s = sm_scale[t][slot];
      if (s != top) {
        // the quotient of an 8-bit and two 24-bit numbers is at least 2^-33 from any half that it
        // does not equal: in 64 bits it rounds as the real number does
        const double f = top > 0.0f ? static_cast<double>(s) / static_cast<double>(top) : 0.0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t o = (&v[i].x)[w];
          uint32_t r = 0;
          if (CODE == kCodeInt8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int k = __double2int_rn(static_cast<double>(code_value<CODE>((o >> (8 * j)) & 0xff)) * f);
              r |= (static_cast<uint32_t>(k) & 0xff) << (8 * j);
            }
          } else {
            const float g = static_cast<float>(f);  // a power of two
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = code_value<CODE>((o >> (8 * j)) & 0xff) * g;
            r = e4m3_pair(x[0], x[1]) | (e4m3_pair(x[2], x[3]) << 16);
          }
          (&v[i].x)[w] = r;
        }
      }
      *reinterpret_cast<uint4*>(p.to.code[t] + (dst * kPage + slot) * D + c) = v[i];
    }
  }
}

}  // namespace

inline cudaError_t launch_paged_evict(const PagedEvictParams& p, int code, cudaStream_t stream) {
  const unsigned heads = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.from.H);
  paged_select_kernel<<<heads, kSelectThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
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
