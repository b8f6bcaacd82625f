// Attention over the paged 8-bit cache for many query rows: tcgen05 MMAs with
// both operands of fp16, scores and outputs in tensor memory.
//
// A work item is up to 256 rows (two tiles of 128, row r = i * G + g as in
// paged_attention.cuh) of one (sequence, key head) against its pages, 128 keys
// (two pages) at a time. One CTA per item and SM, 13 warps:
//   - two softmax warpgroups, one thread per row: query rows to shared memory
//     (bf16 rows times a power of two, exact in fp16), then per key tile the row
//     maximum, 2^(z - R + 7) as fp16 over the scores' own columns, and at the end
//     the output;
//   - four unpack warps: codes straight from global memory into registers one
//     tile ahead, converted (exactly) to fp16 and stored as swizzled K-major
//     tiles, which serve K as they are and V read MN-major;
//   - one MMA warp: S = Q K^T, O += P V (P from tensor memory), ordered so that one
//     tile's products run while the other's softmax does.
// The scales stay out of the operands: K's is a factor of the scores, V's goes into the
// weights as an exponent. A row's reference R covers z + log2(scale_V / v0), v0 the first
// non-zero V scale of the item, and the row sum takes each page's part times v0 / scale_V
// again, so weights keep their 11 bits whatever the pages' scales are (ratios to v0 are
// cut at 2^+-100). R moves only when a row's maximum passes it by 8 (weights reach 2^15);
// the output is then rescaled in tensor memory.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "paged_attention.cuh"

namespace vq {
namespace {

// What the softmax has to do beyond the product: nothing but an interval of slots per
// row; a cap too; or position-dependent terms.
enum ManyMode : int { kManyPlain = 0, kManyCap = 1, kManyGeneral = 2 };

template <int D>
struct ManyCfg {
  static constexpr int KT = 128;
  static constexpr int TILE = 128 * D * 2;  // fp16 [128][D]
  static constexpr int Q0 = 0;
  static constexpr int K0 = 2 * TILE;
  static constexpr int V0 = K0 + 2 * TILE;
  static constexpr int HDR0 = V0 + 2 * TILE;  // 4 x {8 floats, 128 positions}
  static constexpr int HDR = 32 + 128 * 4;
  static constexpr int BARS = HDR0 + 4 * HDR;
  static constexpr int NBARS = 14;
  static constexpr int TMEM_SLOT = BARS + NBARS * 8;
  static constexpr int V0_SLOT = TMEM_SLOT + 8;
  static constexpr int SMEM = V0_SLOT + 8;
  static constexpr int SMEM_ALLOC = SMEM + 1024;
  static constexpr int THREADS = 13 * 32;
  static constexpr int COL_O = 128;  // tile qt: columns 256 * qt: scores [0, 128), output [128, 128 + D)
  static_assert(SMEM_ALLOC <= 232448 && TILE % 1024 == 0, "shared memory");
};

struct ManyRow {
  int lo, hi;   // slots seen (general mode: hi is the causal bound, lo unused)
  int first, pos, prefix;
  float slope;
  bool live;
};

template <int D, int CODE, int MODE>
__global__ void __launch_bounds__(ManyCfg<D>::THREADS, 1) paged_many_kernel(const __grid_constant__ PagedAttnParams p) {
  using C = ManyCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* sm = smem_raw + (sbase - raw);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + C::BARS);
  uint64_t* k_full = q_full + 1;
  uint64_t* k_empty = q_full + 3;
  uint64_t* v_full = q_full + 5;
  uint64_t* v_empty = q_full + 7;
  uint64_t* s_full = q_full + 9;
  uint64_t* p_full = q_full + 11;
  uint64_t* o_full = q_full + 13;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::TMEM_SLOT);
  float* v0_slot = reinterpret_cast<float*>(sm + C::V0_SLOT);
  __shared__ int range[2];  // slots that any row of the item sees

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x % p.splits;
  const int bh = (blockIdx.x / p.splits) % (p.B * p.c.H);
  const int tile = p.row_tiles - 1 - blockIdx.x / (p.splits * p.B * p.c.H);  // longest causal tiles first
  const int b = bh / p.c.H, h = bh - b * p.c.H;
  const int row0 = tile * 256;
  const SeqView sv = seq_view(p, b);
  const int rows = sv.q_len * p.G;
  if (row0 >= rows) return;  // (uniform: no live row)
  const int nq = rows - row0 > 128 ? 2 : 1;

  // ---- set-up
  if (warp == 12) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(q_full, nq * 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 128);
      mbar_init(&v_full[i], 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
    }
    mbar_init(o_full, 1);
    fence_barrier_init();
    range[0] = INT32_MAX;
    range[1] = 0;
    *v0_slot = 1.0f;
  }
  __syncthreads();
  ManyRow rv{};
  if (tid < 256) {
    const RowView r = row_view(p, sv, b, h, row0 + tid);
    rv.live = r.hi >= 0;
    rv.first = r.first;
    rv.pos = r.pos;
    rv.slope = r.slope;
    rv.prefix = p.causal && p.prefix ? sv.prefix : INT32_MIN;
    rv.lo = 0;
    rv.hi = max(r.hi, 0);
    int reach = rv.hi;
    if (rv.live && p.causal && p.prefix) {
      if (MODE == kManyGeneral && p.c.pos)
        reach = sv.len;
      else
        reach = rv.hi = max(rv.hi, min(sv.len, sv.prefix));
    }
    if (!(MODE == kManyGeneral && p.c.pos) && rv.live) rv.lo = max(rv.first, 0);
    int lo = rv.live ? rv.lo : INT32_MAX;
    int hi = rv.live ? reach : 0;
    if (lo >= hi) lo = INT32_MAX, hi = 0;
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      atomicMin(&range[0], lo);
      atomicMax(&range[1], hi);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = *tmem_slot;
  int t0 = 0, T = 0;  // first key tile and number of tiles of this split
  if (range[1] > range[0]) {
    const int first = range[0] / C::KT, all = (range[1] + C::KT - 1) / C::KT - first;
    const int per = (all + p.splits - 1) / p.splits;
    t0 = first + split * per;
    T = max(0, min(all - split * per, per));
  }

  bool ok = true;
  float R = -INFINITY, l = 0.0f;
  if (T == 0) {
    // nothing to see: the rows are written below
  } else if (warp < 8) {
    // ================================================================ softmax
    const int qt = warp >> 2;
    if (qt < nq) {
      const uint32_t lane_tm = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16) + qt * 256;
      float back = 1.0f;
      {  // this thread's query row into the K-major tile
        const int row = row0 + tid;
        const int i = row / p.G, hq = h * p.G + row % p.G;
        const uint4* q = reinterpret_cast<const uint4*>(p.q + b * p.q_sb + hq * p.q_sh + i * p.q_st);
        uint4 v[D / 8];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          v[c] = rv.live ? __ldg(q + c) : make_uint4(0, 0, 0, 0);
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[c].x & 0x7fff7fffu, v[c].y & 0x7fff7fffu),
                                       __vmaxu2(v[c].z & 0x7fff7fffu, v[c].w & 0x7fff7fffu)));
        }
        float f = 1.0f;
        if (p.q_bf16) {
          top = max(top & 0xffffu, top >> 16);
          const int e = max(min(static_cast<int>(top >> 7) - 127, 119), -119);
          f = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23);
          back = __uint_as_float(static_cast<uint32_t>(127 - 7 + e) << 23);
        }
        const int r = tid & 127;
        const uint32_t at = sbase + C::Q0 + qt * C::TILE + (r >> 3) * 1024 + (r & 7) * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          if (p.q_bf16) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t x = (&v[c].x)[w];
              (&v[c].x)[w] = tc::cvt_half2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f);
            }
          }
          tc::sts128(at + (c >> 3) * (128 * 128) + (((c & 7) ^ (r & 7)) << 4), v[c].x, v[c].y, v[c].z, v[c].w);
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
      }
      const float fz = p.sigma * back * (MODE == kManyPlain ? kLog2e : 1.0f);
      const float cap_f = MODE != kManyPlain && p.cap > 0.0f ? 2.0f * kLog2e / p.cap : 0.0f;
      for (int j = 0; j < T; ++j) {
        const int slot0 = (t0 + j) * C::KT;
        ok = mbar_wait_warp(&k_full[j & 1], (j >> 1) & 1) && mbar_wait_warp(&s_full[qt], j & 1);
        if (!ok) break;
        tc::fence_after_sync();
        const float* hdr = reinterpret_cast<const float*>(sm + C::HDR0 + (j & 3) * C::HDR);
        const int* kp = reinterpret_cast<const int*>(hdr + 8);
        const bool with_pos = MODE == kManyGeneral && p.c.pos;
        const int lo = rv.lo - slot0, hi = rv.hi - slot0;
        const bool whole = __all_sync(0xffffffffu, lo <= 0 && hi >= C::KT) && !with_pos;
        // (a page of zero scale still gives -inf where masked)
        const float f0 = fmaxf(hdr[0] * fz, 1e-37f), f1 = fmaxf(hdr[1] * fz, 1e-37f);
        auto seen = [&](int col) {
          if (with_pos) {
            const int k = kp[col];
            return rv.live && slot0 + col < sv.len && (col < hi || k < rv.prefix) && k >= rv.first;
          }
          return col >= lo && col < hi;
        };
        // a score in log2 units, without the mask
        auto score = [&](float a, float f, int col) {
          float z = a * f;
          if (MODE == kManyPlain) return z;
          z = MODE == kManyCap || p.cap > 0.0f ? capped(z, p.cap, cap_f) : z * kLog2e;
          if (MODE == kManyGeneral) {
            const int k = p.c.pos ? kp[col] : slot0 + col;
            z = fmaf(-rv.slope, fabsf(static_cast<float>(rv.pos - k)), z);
          }
          return z;
        };
        float top[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float m = -INFINITY;
#pragma unroll 1
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t a[2][16];
            const int c0 = half * 64 + ch * 32;
            tc::tmem_ld16(lane_tm + c0, a[0]);
            tc::tmem_ld16(lane_tm + c0 + 16, a[1]);
            tc::tmem_wait_ld();
            float x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              x[i] = __uint_as_float(a[i >> 4][i & 15]);
              if (MODE == kManyGeneral) x[i] = score(x[i], half ? f1 : f0, c0 + i);
              if (!whole && !seen(c0 + i)) x[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) m = tc::max3(m, x[i], x[i + 1]);
          }
          // scores grow with the raw products where no bias depends on the key
          if (MODE != kManyGeneral && m > -INFINITY) m = score(m, half ? f1 : f0, 0);
          top[half] = m + hdr[2 + half];
        }
        __syncwarp();
        const float t = fmaxf(top[0], top[1]);
        const bool move = t > R + 8.0f;
        if (__any_sync(0xffffffffu, move)) {
          const float g = move ? tc::ex2(R - t) : 1.0f;
          if (move) R = t;
          l *= g;
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tc::tmem_ld16(lane_tm + C::COL_O + c, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * g);
              tc::tmem_st16(lane_tm + C::COL_O + c, o);
            }
            tc::tmem_wait_st();
          }
        }
        const float base = (R == -INFINITY ? 0.0f : R) - 7.0f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float f = half ? f1 : f0, off = hdr[2 + half] - base;
          uint64_t sum2 = 0;
#pragma unroll 1
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t a[2][16], w[16];
            const int c0 = half * 64 + ch * 32;
            tc::tmem_ld16(lane_tm + c0, a[0]);
            tc::tmem_ld16(lane_tm + c0 + 16, a[1]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float x0 = __uint_as_float(a[i >> 4][i & 15]), x1 = __uint_as_float(a[i >> 4][(i & 15) + 1]);
              if (MODE == kManyPlain) {
                if (!whole) {
                  x0 = seen(c0 + i) ? x0 : -INFINITY;
                  x1 = seen(c0 + i + 1) ? x1 : -INFINITY;
                }
                const uint64_t z = tc::fma2(tc::f2pack(x0, x1), tc::f2pack(f, f), tc::f2pack(off, off));
                x0 = tc::f2lo(z);
                x1 = tc::f2hi(z);
              } else {
                x0 = score(x0, f, c0 + i) + off;
                x1 = score(x1, f, c0 + i + 1) + off;
                if (!whole) {
                  x0 = seen(c0 + i) ? x0 : -INFINITY;
                  x1 = seen(c0 + i + 1) ? x1 : -INFINITY;
                }
              }
              const float p0 = tc::ex2(x0), p1 = tc::ex2(x1);
              sum2 = tc::add2(sum2, tc::f2pack(p0, p1));
              w[i >> 1] = tc::cvt_half2(p0, p1);
            }
            // over columns whose scores this row has read
            tc::tmem_st16(lane_tm + half * 32 + ch * 16, w);
          }
          l = fmaf(tc::f2lo(sum2) + tc::f2hi(sum2), hdr[4 + half], l);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        mbar_arrive(&p_full[qt]);
      }
    }
  } else if (warp < 12) {
    // ================================================================= unpack
    constexpr int G = D / 16, N = D / 16, RPI = 128 / G;  // 16-code groups per row, loads per thread, rows per load
    const int u = tid - 256;
    const int g = u % G, r0 = u / G;
    const int last = (sv.len + kPage - 1) / kPage;  // pages that hold tokens
    uint4 kr[N], vr[N];
    int64_t ph[2];     // (page * H + h) of the tile's two pages, -1: none
    float ks[2], vs[2];
    int pos = 0;
    float v0 = 0.0f;
    auto locate = [&](int j) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int index = (t0 + j) * 2 + i;
        const int page = index < last ? paged_page(p.c, b, index) : -1;
        ph[i] = page < 0 ? -1 : static_cast<int64_t>(page) * p.c.H + h;
      }
    };
    auto load = [&](const unsigned char* code, const int64_t (&at)[2], uint4 (&x)[N]) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = (i * RPI + r0) & 63;
        const int64_t a = at[i >= N / 2];
        x[i] = a < 0 ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4*>(code + (a * kPage + row) * D + g * 16));
      }
    };
    auto store = [&](const uint4 (&x)[N], uint32_t dst) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = i * RPI + r0;
        const uint32_t at = dst + (g >> 2) * (128 * 128) + (row >> 3) * 1024 + (row & 7) * 128;
        uint32_t y[8];
        codes_f16<CODE>(x[i].x, y[0], y[1]);
        codes_f16<CODE>(x[i].y, y[2], y[3]);
        codes_f16<CODE>(x[i].z, y[4], y[5]);
        codes_f16<CODE>(x[i].w, y[6], y[7]);
        const uint32_t c0 = (g & 3) * 2;
        // (the second 64 channels' lanes store their odd chunk first: eight lanes then cover all banks)
        const bool odd = (g >> 2) & 1;
        tc::sts128(at + (((c0 + odd) ^ (row & 7)) << 4), odd ? y[4] : y[0], odd ? y[5] : y[1], odd ? y[6] : y[2],
                   odd ? y[7] : y[3]);
        tc::sts128(at + (((c0 + 1 - odd) ^ (row & 7)) << 4), odd ? y[0] : y[4], odd ? y[1] : y[5], odd ? y[2] : y[6],
                   odd ? y[3] : y[7]);
      }
    };
    auto scales = [&]() {
      if (u == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ks[i] = ph[i] < 0 ? 0.0f : __ldg(p.c.scale[0] + ph[i]);
          vs[i] = ph[i] < 0 ? -1.0f : __ldg(p.c.scale[1] + ph[i]);
        }
      }
      if (MODE == kManyGeneral && p.c.pos) pos = ph[u >> 6] < 0 ? 0 : __ldg(p.c.pos + ph[u >> 6] * kPage + (u & 63));
    };
    locate(0);
    scales();
    load(p.c.code[0], ph, kr);
    load(p.c.code[1], ph, vr);
    for (int j = 0; j < T; ++j) {
      if (j >= 2 && !(ok = mbar_wait_warp(&k_empty[j & 1], ((j >> 1) - 1) & 1))) break;
      store(kr, sbase + C::K0 + (j & 1) * C::TILE);
      // header of the tile; its slot was last read by the softmax of tile j - 4, which tile j - 2's products follow
      float* hdr = reinterpret_cast<float*>(sm + C::HDR0 + (j & 3) * C::HDR);
      if (u == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          hdr[i] = ks[i] * code_unit<CODE>();
          float lc = 0.0f, inv = 1.0f;
          if (vs[i] < 0.0f) {
            lc = -INFINITY;  // no such page: its keys have no weight
          } else if (vs[i] > 0.0f) {
            if (v0 == 0.0f) *v0_slot = v0 = vs[i];
            const float c = fminf(fmaxf(__fdiv_rn(vs[i], v0), 7.888609052210118e-31f), 1.2676506002282294e30f);
            lc = log2f(c);
            inv = __fdiv_rn(1.0f, c);
          }
          hdr[2 + i] = lc;
          hdr[4 + i] = inv;
        }
      }
      if (MODE == kManyGeneral && p.c.pos) reinterpret_cast<int*>(hdr + 8)[u] = pos;
      fence_proxy_async_smem();
      mbar_arrive(&k_full[j & 1]);
      if (j + 1 < T) {
        locate(j + 1);
        scales();
        load(p.c.code[0], ph, kr);
      }
      if (j >= 2 && !(ok = mbar_wait_warp(&v_empty[j & 1], ((j >> 1) - 1) & 1))) break;
      store(vr, sbase + C::V0 + (j & 1) * C::TILE);
      fence_proxy_async_smem();
      mbar_arrive(&v_full[j & 1]);
      if (j + 1 < T) load(p.c.code[1], ph, vr);
    }
  } else {
    // ==================================================================== MMA
    const uint32_t idesc_qk = tc::idesc_f16_f32(128, 128);
    const uint32_t idesc_pv = tc::idesc_f16_f32(128, D, /*b_mn_major=*/true);
    const uint64_t qd = tc::sw128_desc(sbase + C::Q0);
    const uint64_t kd = tc::sw128_desc(sbase + C::K0);
    const uint64_t vd = tc::sw128_desc_mn(sbase + C::V0, 128 * 128);
    auto qk = [&](int qt, int slot) {
      const uint64_t a = qd + static_cast<uint64_t>((qt * C::TILE) >> 4), bq = kd + static_cast<uint64_t>((slot * C::TILE) >> 4);
#pragma unroll 1
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t o = static_cast<uint64_t>(((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4);
        tc::mma_f16_ss_warp(tm + qt * 256, a + o, bq + o, idesc_qk, kk > 0 ? 1u : 0u);
      }
    };
    auto pv = [&](int qt, int slot, bool first) {
      const uint64_t bv = vd + static_cast<uint64_t>((slot * C::TILE) >> 4);
#pragma unroll 1
      for (int kk = 0; kk < 8; ++kk)
        tc::mma_f16_ts_warp(tm + qt * 256 + C::COL_O, tm + qt * 256 + 8 * kk, bv + static_cast<uint64_t>((kk * 2048) >> 4),
                            idesc_pv, (first && kk == 0) ? 0u : 1u);
    };
    ok = mbar_wait_warp(q_full, 0);
    for (int j = 0; ok && j < T; ++j) {
      const int s = j & 1;
      if (!(ok = mbar_wait_warp(&k_full[s], (j >> 1) & 1))) break;
      tc::fence_after_sync();
      qk(0, s);
      tc::commit_warp(&s_full[0]);
      if (nq == 2) {
        if (j > 0) {
          if (!(ok = mbar_wait_warp(&p_full[1], (j - 1) & 1))) break;
          tc::fence_after_sync();
          pv(1, s ^ 1, j == 1);
          tc::commit_warp(&v_empty[s ^ 1]);
        }
        qk(1, s);
        tc::commit_warp(&s_full[1]);
      }
      tc::commit_warp(&k_empty[s]);
      if (!(ok = mbar_wait_warp(&v_full[s], (j >> 1) & 1) && mbar_wait_warp(&p_full[0], j & 1))) break;
      tc::fence_after_sync();
      pv(0, s, j == 0);
      if (nq == 1) tc::commit_warp(&v_empty[s]);
    }
    if (ok && nq == 2 && (ok = mbar_wait_warp(&p_full[1], (T - 1) & 1))) {
      tc::fence_after_sync();
      pv(1, (T - 1) & 1, T == 1);
    }
    if (ok) tc::commit_warp(o_full);
  }

  // ---- output: one row per thread
  if (warp < 8 && (warp >> 2) < nq) {
    const uint32_t lane_tm = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (warp >> 2) * 256 + C::COL_O;
    if (T > 0) {
      ok = ok && mbar_wait_warp(o_full, 0);
      tc::fence_after_sync();
    }
    const int row = row0 + tid;
    const int i = row / p.G, hq = h * p.G + row % p.G;
    const bool part = p.splits > 1;
    const float v0 = *v0_slot * code_unit<CODE>();
    const float inv = part ? v0 : (l == 0.0f ? 0.0f : __fdiv_rn(v0, l));
    const int64_t pr = (static_cast<int64_t>(split) * p.B * p.c.H + bh) * (static_cast<int64_t>(p.row_tiles) * 256) + row;
#pragma unroll 1
    for (int c = 0; ok && c < D; c += 16) {
      uint32_t o[16];
      if (T > 0) {
        tc::tmem_ld16(lane_tm + c, o);
        tc::tmem_wait_ld();
      } else {
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = 0;
      }
      float v[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) v[x] = __uint_as_float(o[x]) * inv;
      if (!rv.live) {
        // a row of no query is left as it is
      } else if (part) {
#pragma unroll
        for (int x = 0; x < 16; x += 4)
          *reinterpret_cast<float4*>(p.part_o + pr * D + c + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
      } else {
        uint32_t w[8];
#pragma unroll
        for (int x = 0; x < 8; ++x)
          w[x] = p.q_bf16 ? tc::cvt_bf162(v[2 * x], v[2 * x + 1]) : tc::cvt_half2(v[2 * x], v[2 * x + 1]);
        uint4* out = reinterpret_cast<uint4*>(p.out + b * p.o_sb + hq * p.o_sh + i * p.o_st + c);
        out[0] = make_uint4(w[0], w[1], w[2], w[3]);
        out[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
      __syncwarp();
    }
    if (ok && rv.live) {
      if (part)
        p.part_ml[pr] = make_float2(R, l);
      else if (p.lse)
        p.lse[(static_cast<int64_t>(b) * p.Hq + hq) * p.n + i] = l == 0.0f ? -INFINITY : (R - 7.0f + log2f(l)) * kLn2;
    }
    tc::fence_before_sync();
  }
  __syncthreads();
  if (warp == 12) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tm, 512);
  }
}

template <int D, int CODE, int MODE>
cudaError_t launch_many_variant(const PagedAttnParams& p, unsigned grid, cudaStream_t stream) {
  using C = ManyCfg<D>;
  static bool configured[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(paged_many_kernel<D, CODE, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  paged_many_kernel<D, CODE, MODE><<<grid, C::THREADS, C::SMEM_ALLOC, stream>>>(p);
  return cudaGetLastError();
}

inline cudaError_t launch_paged_many(const PagedAttnParams& p, int code, unsigned grid, cudaStream_t stream) {
  const bool general = p.slopes || (p.c.pos && (p.first || (p.prefix && p.causal)));
  auto by_mode = [&](auto d, auto c) {
    if (general) return launch_many_variant<d(), c(), kManyGeneral>(p, grid, stream);
    if (p.cap > 0.0f) return launch_many_variant<d(), c(), kManyCap>(p, grid, stream);
    return launch_many_variant<d(), c(), kManyPlain>(p, grid, stream);
  };
  auto by_code = [&](auto d) {
    return code == kCodeInt8 ? by_mode(d, std::integral_constant<int, kCodeInt8>{})
                             : by_mode(d, std::integral_constant<int, kCodeE4m3>{});
  };
  return p.c.D == 64 ? by_code(std::integral_constant<int, 64>{}) : by_code(std::integral_constant<int, 128>{});
}

}  // namespace
}  // namespace vq
