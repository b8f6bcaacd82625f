// Sums of the attention weights per cached token, for many query rows: the scores
// transposed, one tcgen05 product per 128 keys and 128 rows, so that a thread owns a
// key (its tensor-memory lane) and sums along its columns: no atomics, no reduction
// between threads, results that repeat to the bit.
//
// One CTA per 128 cached tokens (two pages) of a (sequence, key head), two CTAs per SM.
// Its K codes are converted once, exactly, to the queries' own type, so the query rows go
// to shared memory as they are. Nine warps: four copy rows (and what a row sees and its
// log-sum-exp) into a ring of two, one issues the products into two score buffers, four
// read them: w += 2^(z log2 e - lse log2 e). 1560 queries over 18720 tokens, 2 x 12 heads: 363 us, where the
// exponentials (16 a clock and SM) take 164 and the products 106.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged_many.cuh"

namespace vq {
namespace {

// The four codes of a word as two bf16x2, exactly.
template <int CODE>
__device__ __forceinline__ uint32_t code_pair_bf16(uint32_t w, int pair) {
  if (CODE == kCodeInt8) {
    // 128 + low seven bits, minus 128 (or 256 for a set sign bit)
    const uint32_t v = __byte_perm(w, 0x43434343u, pair ? 0x4342 : 0x4140);
    const uint32_t a = v & 0xff7fff7fu, b = v & 0xff80ff80u;
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  // exponent and mantissa bits in place, 2^-120 times the value, subnormals included
  const uint32_t v = __byte_perm(w, 0u, pair ? 0x3424 : 0x1404);
  const uint32_t a = (v & 0x80008000u) | ((v & 0x7f007f00u) >> 4);
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), __bfloat162bfloat162(__ushort_as_bfloat16(0x7b80)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int D>
struct SumCfg {
  static constexpr int TILE = 128 * D * 2;
  static constexpr int K0 = 0;
  static constexpr int Q0 = TILE;               // ring of two
  static constexpr int META0 = 3 * TILE;        // ring of five SumRows
  static constexpr int META = 128 * 20 + 16;
  static constexpr int AT0 = META0 + 5 * META;  // the rows' places in q, in elements, -1: none (two tiles)
  static constexpr int BARS = AT0 + 2 * 128 * 8;
  static constexpr int NBARS = 13;
  static constexpr int TMEM_SLOT = BARS + NBARS * 8;
  static constexpr int SMEM = TMEM_SLOT + 16;
  static constexpr int SMEM_ALLOC = SMEM + 1024;
  static constexpr int THREADS = 9 * 32;
  static_assert(META0 % 16 == 0 && META % 16 == 0, "alignment");
  static_assert(2 * SMEM_ALLOC <= 232448 - 2048, "two CTAs per SM");
};

struct SumRows {
  float lse[128];   // log2 units; +inf: no weight
  float slope[128];
  int hi[128];      // slots seen are [lo, hi) (where positions decide: hi the causal bound, lo the first position)
  int lo[128];
  float pos[128];   // from the first query's
  int whole[4];     // whether every row of 32 sees the whole key tile
};

template <int D, int CODE, int MODE>
__global__ void __launch_bounds__(SumCfg<D>::THREADS, 2) paged_sums_kernel(const __grid_constant__ PagedAttnParams p) {
  using C = SumCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* sm = smem_raw + (sbase - raw);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + C::BARS);
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_full + 4;
  uint64_t* s_empty = q_full + 6;
  uint64_t* m_full = q_full + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::TMEM_SLOT);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = (p.c.max_pages + 1) / 2;
  const int bh = blockIdx.x / groups;
  const int b = bh / p.c.H, h = bh - b * p.c.H;
  const int slot0 = (blockIdx.x % groups) * 128;
  const SeqView sv = seq_view(p, b);
  if (slot0 >= sv.len) return;  // (uniform)
  int64_t ph[2];
  many_pages(p, sv, b, h, slot0 / kPage, ph);
  const int rows = sv.q_len * p.G;
  const bool with_pos = MODE == kGeneral && p.c.pos;
  const bool by_pos = with_pos && (p.first || (p.prefix && p.causal));  // positions decide what is seen
  int rt0 = 0;
  // row tiles that end before the causal rule lets any of their rows see this tile (a prefix may let every row)
  if (p.causal && !(p.prefix && (p.c.pos || slot0 < sv.prefix)))
    rt0 = static_cast<int>(min(static_cast<int64_t>(max(0, slot0 - (sv.len - sv.q_len))) * p.G / 128, int64_t(1) << 30));
  const int T = max(0, (rows + 127) / 128 - rt0);

  if (warp == 8) {
    tc::tmem_alloc(tmem_slot, 256);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    for (int i = 0; i < 5; ++i) mbar_init(&m_full[i], 4);
    fence_barrier_init();
  }
  if (warp < 8) {  // K, once
    constexpr int RPW = 512 / D, N = 128 / RPW / 8;
    int r0, g;
    unpack_lane<D>(lane, r0, g);
    r0 += warp * RPW;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = i * 8 * RPW + r0;
      const int64_t a = row < 64 ? ph[0] : ph[1];
      const uint4 x = a < 0 ? make_uint4(0, 0, 0, 0)
                            : __ldg(reinterpret_cast<const uint4*>(p.c.code[0] + (a * kPage + (row & 63)) * D + g * 16));
      const uint32_t at = sbase + C::K0 + unpack_at(row, g);
      if (p.q_bf16) {
        uint32_t y[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) y[w] = code_pair_bf16<CODE>((&x.x)[w >> 1], w & 1);
        tc::sts128(at, y[0], y[1], y[2], y[3]);
        tc::sts128(at ^ 16u, y[4], y[5], y[6], y[7]);
      } else {
        store_codes<CODE>(x, at);
      }
    }
    fence_proxy_async_smem();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = *tmem_slot;

  bool ok = true;
  if (warp < 4) {
    // ====================================================== one key per thread
    const int64_t a = tid < 64 ? ph[0] : ph[1];
    const int slot = slot0 + tid;
    const bool key = a >= 0 && slot < sv.len;
    const float unit = p.q_bf16 ? 1.0f : code_unit<CODE>();
    const float f = a < 0 ? 0.0f : __ldg(p.c.scale[0] + a) * p.sigma * unit * (MODE == kPlain ? kLog2e : 1.0f);
    const float cap_f = MODE != kPlain && p.cap > 0.0f ? 2.0f * kLog2e / p.cap : 0.0f;
    const int kp = with_pos ? (key ? __ldg(p.c.pos + a * kPage + (tid & 63)) : 0) : slot;
    const float kf = static_cast<float>(kp - sv.pos0);
    const bool cap = MODE == kCap || (MODE == kGeneral && p.cap > 0.0f);
    const float over = cap ? 1.0f / p.cap : 0.0f;
    const uint32_t lane_tm = tm + (static_cast<uint32_t>(warp * 32) << 16);
    const int prefix = p.causal && p.prefix ? sv.prefix : INT32_MIN;
    float w = 0.0f;
    int slot_m = 0, turn_m = 0;  // ring of five: slot, and the parity of its use
    for (int j = 0; j < T; ++j) {
      ok = mbar_wait_warp(&m_full[slot_m], turn_m) && mbar_wait_warp(&s_full[j & 1], (j >> 1) & 1);
      if (!ok) break;
      tc::fence_after_sync();
      const SumRows& meta = *reinterpret_cast<const SumRows*>(sm + C::META0 + slot_m * C::META);
      if (++slot_m == 5) slot_m = 0, turn_m ^= 1;
      const int4 whole4 = *reinterpret_cast<const int4*>(meta.whole);
      const bool whole = whole4.x & whole4.y & whole4.z & whole4.w;
      float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll 1
      for (int c0 = 0; c0 < 128; c0 += 32) {
        float x[32];
        __syncwarp();  // (tensor memory wants the warp as one)
        tmem_ld32(lane_tm + (j & 1) * 128 + c0, x);
        float4 ls[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) ls[i] = *reinterpret_cast<const float4*>(&meta.lse[c0 + 4 * i]);
        tc::tmem_wait_ld();
        bool small = false;
        if (cap) {
          float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            m0 = tc::max3(m0, fabsf(x[i]), fabsf(x[i + 1]));
            m1 = tc::max3(m1, fabsf(x[i + 2]), fabsf(x[i + 3]));
          }
          small = __all_sync(0xffffffffu, fmaxf(m0, m1) * f <= kCapSmall * p.cap);
        }
        if (MODE != kPlain) {
          if (small) {
            const float fc = f * over, cl = p.cap * kLog2e;
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = capped_small(x[i], fc, cl);
          } else if (cap) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = capped(x[i] * f, p.cap, over, cap_f);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] *= f * kLog2e;
          }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float z = MODE == kPlain ? x[i] * f : x[i];
          if (MODE == kGeneral) z = fmaf(-meta.slope[c0 + i], fabsf(meta.pos[c0 + i] - kf), z);
          z -= (&ls[i >> 2].x)[i & 3];
          if (!whole) {
            const int hi = meta.hi[c0 + i], lo = meta.lo[c0 + i];
            const bool see = by_pos ? (slot < hi || kp < prefix) && kp >= lo : slot < hi && slot >= lo;
            z = see ? z : -INFINITY;
          }
          const float e = tc::ex2(z);
          if (i & 1)
            sum1 += e;
          else
            sum0 += e;
        }
      }
      w += sum0 + sum1;
      tc::fence_before_sync();
      warp_arrive(&s_empty[j & 1], lane);
    }
    if (ok && key) {
      float* at = p.c.weight + a * kPage + (tid & 63);
      *at = p.accumulate ? *at + w : w;
    }
  } else if (warp < 8) {
    // ================================================================ row copies
    const int u = tid - 128;
    constexpr int CPR = D / 8, RPI = 128 / CPR;  // 16-byte chunks per row, rows per pass of the four warps
    auto full = [&](int j) {
      fence_proxy_async_smem();
      warp_arrive(&q_full[j & 1], lane);
    };
    int64_t* ats = reinterpret_cast<int64_t*>(sm + C::AT0);
    // what this thread's row of a tile sees, loaded a tile ahead
    RowView v;
    int64_t at;
    float lse;
    auto look = [&](int j) {
      const int row = (rt0 + j) * 128 + u;
      v = row_view(p, sv, b, h, row);
      at = -1;
      lse = -INFINITY;
      if (v.hi >= 0) {
        const int i = row / p.G, hq = h * p.G + row % p.G;
        lse = __ldg(p.lse + (static_cast<int64_t>(b) * p.Hq + hq) * p.n + i);
        if (lse != -INFINITY) at = b * p.q_sb + hq * p.q_sh + i * p.q_st;  // (a row that saw nothing: zeros, whatever its bytes)
      }
    };
    if (T > 0) look(0);
    int slot_m = 0;
    for (int j = 0; j < T; ++j) {
      // (after a wait that gave up, the four warps still meet at every barrier below; the ring's slot was last read with
      // the scores of tile j - 5, and the products of tile j - 3, waited for a turn ago, follow those)
      SumRows& meta = *reinterpret_cast<SumRows*>(sm + C::META0 + slot_m * C::META);
      uint64_t* full_m = &m_full[slot_m];
      if (++slot_m == 5) slot_m = 0;
      {
        int lo, hi;
        row_interval(p, sv, v, by_pos, lo, hi);
        if (by_pos) lo = v.first;
        const bool none = v.hi < 0 || lse == -INFINITY;
        meta.lse[u] = none ? INFINITY : lse * kLog2e;
        meta.slope[u] = v.slope;
        meta.hi[u] = hi;
        meta.lo[u] = lo;
        meta.pos[u] = v.pos;
        ats[(j & 1) * 128 + u] = at;
        const bool all = __all_sync(0xffffffffu, none || (!by_pos && lo <= slot0 && hi >= slot0 + 128));
        if (lane == 0) meta.whole[warp - 4] = all;
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (!ok) continue;
      warp_arrive(full_m, lane);
      if (j + 1 < T) look(j + 1);
      if (j >= 2 && !(ok = mbar_wait_warp(&q_empty[j & 1], ((j >> 1) - 1) & 1))) continue;
      const int c = u % CPR;
      const uint32_t to = sbase + C::Q0 + (j & 1) * C::TILE + (c >> 3) * (128 * 128);
#pragma unroll
      for (int i = 0; i < 128 / RPI; ++i) {
        const int row = i * RPI + u / CPR;
        const int64_t at = ats[(j & 1) * 128 + row];
        copy16_or_zero(to + (row >> 3) * 1024 + (row & 7) * 128 + (((c & 7) ^ (row & 7)) << 4),
                       p.q + (at < 0 ? 0 : at + c * 8), at >= 0);
      }
      copy_commit();
      if (j > 0) {
        copy_wait<1>();
        full(j - 1);
      }
    }
    copy_wait<0>();
    if (ok && T > 0) full(T - 1);
  } else {
    // ======================================================================= MMA
    const uint32_t idesc = tc::idesc_f16_f32(128, 128, false, p.q_bf16 != 0);
    const uint64_t kd = tc::sw128_desc(sbase + C::K0);
    const uint64_t qd = tc::sw128_desc(sbase + C::Q0);
    for (int j = 0; j < T; ++j) {
      const int s = j & 1;
      ok = mbar_wait_warp(&q_full[s], (j >> 1) & 1) && (j < 2 || mbar_wait_warp(&s_empty[s], ((j >> 1) - 1) & 1));
      if (!ok) break;
      tc::fence_after_sync();
      const uint64_t bq = qd + static_cast<uint64_t>((s * C::TILE) >> 4);
#pragma unroll 1
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t o = static_cast<uint64_t>(((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4);
        tc::mma_f16_ss_warp(tm + s * 128, kd + o, bq + o, idesc, kk > 0 ? 1u : 0u);
      }
      tc::commit_warp(&s_full[s]);
      tc::commit_warp(&q_empty[s]);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tm, 256);
  }
}

}  // namespace
}  // namespace vq
