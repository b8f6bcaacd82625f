// Attention over the paged 8-bit cache for many query rows: tcgen05 MMAs with
// both operands of fp16, scores and outputs in tensor memory.
//
// A work item is up to 256 rows (two tiles of 128, row r = i * G + g as in
// paged_attention.cuh) of one (sequence, key head) against its pages, 128 keys
// (two pages) at a time. One CTA per item and SM:
//   - two softmax warpgroups, one thread per row: query rows to shared memory
//     (bf16 rows times a power of two, as fp16), then per key tile the row
//     maximum, 2^(z - R + 7) as fp16 over the scores' own columns, and at the end
//     the output;
//   - four warps unpack K and three V: codes straight from global memory into
//     registers one tile ahead, converted (exactly) to fp16 and stored as swizzled
//     K-major tiles, which serve K as they are and V read MN-major;
//   - one MMA warp: S = Q K^T, O += P V (P from tensor memory), ordered so that one
//     tile's products run while the other's softmax does.
// The scales stay out of the operands: K's is a factor of the scores, V's goes into the
// weights as an exponent, c = log2(scale_V / v0), v0 the first non-zero V scale of the item
// (-inf for a page of zeros). A row has two references, so that both its output and its sum
// keep their bits however far apart the pages' scales are: R covers z + c, the output's, and
// L covers z, the sum's. A page's part of the sum is that of its weights, 2^(z + c - R + 7),
// times 2^(R - c - L); a weight's exponent goes no lower than z - L - 53, where the weight is
// zero in fp16 (at most 2^-45) and still counts in the sum. A reference moves only when a
// row's maximum passes it by 8 (weights reach 2^15); the output is then rescaled in tensor
// memory. (One reference and ratios cut at 2^+-100 took 935 us where two take 962, below.)
//
// 2 x 16 heads of 4096 queries over 10521 tokens: 962 us, 734 TFLOP/s. A period of 256 rows
// and 128 keys takes about 5050 cycles; its products take 2240 and its exponentials 2050.
// What sets it is each query tile's chain (scores, softmax, P V, the next scores: P lies
// over S, for which tensor memory has no second place at head_dim 128). A unit of 128 rows
// would unpack K and V twice as often. (Its 512 items are 3.46 waves of the 148 SMs and run as
// 4: 13 % of the SMs' time is idle.)
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "paged_attention.cuh"

namespace vq {
namespace {

// A row's references before it has seen a score: below every score, and finite, so that no sum of them is a NaN.
constexpr float kNoScore = -3e38f;

template <int D>
struct ManyCfg {
  static constexpr int KT = 128;
  static constexpr int TILE = 128 * D * 2;  // fp16 [128][D]
  static constexpr int Q0 = 0;
  static constexpr int K0 = 2 * TILE;
  static constexpr int V0 = K0 + 2 * TILE;
  static constexpr int HDR0 = V0 + 2 * TILE;  // 4 x {8 floats, 128 x {position, the same from the first query's, float32}}
  static constexpr int HDR = 32 + 128 * 8;
  static constexpr int BARS = HDR0 + 4 * HDR;
  static constexpr int NBARS = 18;
  static constexpr int TMEM_SLOT = BARS + NBARS * 8;
  static constexpr int V0_SLOT = TMEM_SLOT + 8;
  static constexpr int SMEM = V0_SLOT + 8;
  static constexpr int SMEM_ALLOC = SMEM + 1024;
  static constexpr int THREADS = 512;  // 128 registers each at launch, shared out below: 256 x 152 + 128 x 80 + 128 x 128
  static constexpr int COL_O = 128;  // tile qt: columns 256 * qt: scores [0, 128), output [128, 128 + D)
  static_assert(SMEM_ALLOC <= 232448 && TILE % 1024 == 0, "shared memory");
};

// Thread t of the warp reads TMEM lane (base + t), 32 consecutive 32-bit columns; not waited for.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* x) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
}

// One arrival for the whole warp, after all of its lanes' work.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// The registers of this warpgroup's threads from here on.
template <int N>
__device__ __forceinline__ void set_registers() {
  if constexpr (N > 128)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// (page * H + h) of pages index and index + 1 of sequence b; -1 where no token is, or the page id is out of range.
__device__ __forceinline__ void many_pages(const PagedAttnParams& p, const SeqView& sv, int b, int h, int index,
                                           int64_t (&ph)[2]) {
  const int last = (sv.len + kPage - 1) / kPage;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int page = index + i < last ? paged_page(p.c, b, index + i) : -1;
    ph[i] = page < 0 ? -1 : static_cast<int64_t>(page) * p.c.H + h;
  }
}

// Which row (of the warp load's 128 / D * 4) and which 16 codes of it a lane takes: a quarter of the warp takes 64
// channels of two rows, so that its 16-byte stores cover all banks (chunks 0, 2, 4, 6 of one row and 1, 3, 5, 7 of
// the next, under the swizzle).
template <int D>
__device__ __forceinline__ void unpack_lane(int lane, int& row, int& g) {
  const int quarter = lane >> 3;
  row = (D == 128 ? (quarter >> 1) * 2 : quarter * 2) + ((lane >> 2) & 1);
  g = (D == 128 ? (quarter & 1) * 4 : 0) + (lane & 3);
}
// Byte offset of row `row`, 16-code group g in the K-major 128-byte-swizzled fp16 tile of 128 rows: its first 16
// bytes; the other 16 are at the offset xor 16.
__device__ __forceinline__ uint32_t unpack_at(int row, int g) {
  return (g >> 2) * (128 * 128) + (row >> 3) * 1024 + (row & 7) * 128 + ((((g & 3) * 2) ^ (row & 7)) << 4);
}
template <int CODE>
__device__ __forceinline__ void store_codes(const uint4& x, uint32_t at) {
  uint32_t y[8];
  codes_f16<CODE>(x.x, y[0], y[1]);
  codes_f16<CODE>(x.y, y[2], y[3]);
  codes_f16<CODE>(x.z, y[4], y[5]);
  codes_f16<CODE>(x.w, y[6], y[7]);
  tc::sts128(at, y[0], y[1], y[2], y[3]);
  tc::sts128(at ^ 16u, y[4], y[5], y[6], y[7]);
}

// Query i and head g (of its key head's) of a row, and of rows a fixed step further on, without a division for each.
struct RowWalk {
  int i, g, di, dg;
  __device__ __forceinline__ RowWalk(const PagedAttnParams& p, int row, int step)
      : i(row / p.G), g(row % p.G), di(step / p.G), dg(step % p.G) {}
  __device__ __forceinline__ void next(const PagedAttnParams& p) {
    i += di;
    g += dg;
    if (g >= p.G) g -= p.G, ++i;
  }
};

struct ManyRow {
  int lo, hi;  // slots seen (where positions decide: hi is the causal bound, lo unused)
  int first, prefix;
  float pos, slope;
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
  uint64_t* h_full = q_full + 14;  // four headers
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

  // the query rows into their K-major tiles as they are, whole rows at a time, by all warps; what follows hides their way
  {
    constexpr int CPR = D / 8, RPI = 512 / CPR;  // 16-byte chunks per row, rows per pass of the CTA
    const int c = tid % CPR;
    const uint16_t* q = p.q + b * p.q_sb + static_cast<int64_t>(h) * p.G * p.q_sh + c * 8;
    RowWalk at(p, row0 + tid / CPR, RPI);
    int r = tid / CPR;
#pragma unroll 4
    for (int x = 0; x < 256 / RPI; ++x, r += RPI, at.next(p)) {
      const bool live = at.i < sv.q_len;
      copy16_or_zero(sbase + C::Q0 + (r >> 7) * C::TILE + (c >> 3) * (128 * 128) + ((r & 127) >> 3) * 1024 + (r & 7) * 128 +
                         (((c & 7) ^ (r & 7)) << 4),
                     q + (live ? at.g * p.q_sh + at.i * p.q_st : 0), live);
    }
    copy_commit();
  }

  // ---- set-up
  if (warp == 15) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(q_full, nq * 4);  // (one arrival per warp)
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 4);
      mbar_init(&v_full[i], 3);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
    }
    mbar_init(o_full, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&h_full[i], 4);
    fence_barrier_init();
    range[0] = INT32_MAX;
    range[1] = 0;
    *v0_slot = 1.0f;
  }
  __syncthreads();
  const bool with_pos = MODE == kGeneral && p.c.pos;
  const bool by_pos = with_pos && (p.first || (p.prefix && p.causal));  // positions decide what is seen
  ManyRow rv{};
  if (tid < 256) {
    const RowView r = row_view(p, sv, b, h, row0 + tid);
    rv.live = r.hi >= 0;
    rv.first = r.first;
    rv.pos = r.pos;
    rv.slope = r.slope;
    rv.prefix = p.causal && p.prefix ? sv.prefix : INT32_MIN;
    row_interval(p, sv, r, by_pos, rv.lo, rv.hi);
    const int reach = by_pos && rv.live && p.causal && p.prefix ? sv.len : rv.hi;
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
  copy_wait<0>();
  fence_proxy_async_smem();
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
  float R = kNoScore, L = kNoScore, l = 0.0f;  // references of the output and of the sum, and the sum
  if (T == 0) {
    // nothing to see: the rows are written below
  } else if (warp < 8) {
    // ================================================================ softmax
    set_registers<152>();
    const int qt = warp >> 2;
    if (qt < nq) {
      const uint32_t lane_tm = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16) + qt * 256;
      float back = 1.0f;
      {  // bf16 rows to fp16 in place
        constexpr int CPR = D / 8, RPI = 32 / CPR, N = 32 / RPI;  // 16-byte chunks per row, rows at a time, turns
        constexpr int U = 4;
        const int c = lane % CPR;
        if (p.q_bf16) {
#pragma unroll 1
          for (int x0 = 0; x0 < N; x0 += U) {
            uint4 v[U];
            uint32_t top[U], place[U];
#pragma unroll
            for (int x = 0; x < U; ++x) {
              const int r = (warp & 3) * 32 + (x0 + x) * RPI + lane / CPR;
              place[x] = C::Q0 + qt * C::TILE + (c >> 3) * (128 * 128) + (r >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4);
              v[x] = lds128(sm + place[x]);
            }
#pragma unroll
            for (int x = 0; x < U; ++x) {
              const uint32_t m = __vmaxu2(__vmaxu2(v[x].x & 0x7fff7fffu, v[x].y & 0x7fff7fffu),
                                          __vmaxu2(v[x].z & 0x7fff7fffu, v[x].w & 0x7fff7fffu));
              top[x] = max(m & 0xffffu, m >> 16);
            }
#pragma unroll
            for (int o = 1; o < CPR; o <<= 1)
#pragma unroll
              for (int x = 0; x < U; ++x) top[x] = max(top[x], __shfl_xor_sync(0xffffffffu, top[x], o));
#pragma unroll
            for (int x = 0; x < U; ++x) {
              const int e = max(min(static_cast<int>(top[x] >> 7) - 127, 119), -119);
              const float f = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23);
              const int e_mine = __shfl_sync(0xffffffffu, e, (lane % RPI) * CPR);  // of row (x0 + x) * RPI + lane % RPI
              if (lane / RPI == x0 + x) back = __uint_as_float(static_cast<uint32_t>(127 - 7 + e_mine) << 23);
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t y = (&v[x].x)[w];
                (&v[x].x)[w] = tc::cvt_half2(__uint_as_float(y << 16) * f, __uint_as_float(y & 0xffff0000u) * f);
              }
              tc::sts128(sbase + place[x], v[x].x, v[x].y, v[x].z, v[x].w);
            }
          }
        }
        fence_proxy_async_smem();
        warp_arrive(q_full, lane);
      }
      const float fz = p.sigma * back * (MODE == kPlain ? kLog2e : 1.0f);
      const float cap_f = MODE != kPlain && p.cap > 0.0f ? 2.0f * kLog2e / p.cap : 0.0f;
      const float over = MODE != kPlain && p.cap > 0.0f ? 1.0f / p.cap : 0.0f;
      for (int j = 0; j < T; ++j) {
        const int slot0 = (t0 + j) * C::KT;
        ok = mbar_wait_warp(&h_full[j & 3], (j >> 2) & 1) && mbar_wait_warp(&s_full[qt], j & 1);
        if (!ok) break;
        tc::fence_after_sync();
        const float* hdr = reinterpret_cast<const float*>(sm + C::HDR0 + (j & 3) * C::HDR);
        const int2* kp = reinterpret_cast<const int2*>(hdr + 8);
        const int lo = rv.lo - slot0, hi = rv.hi - slot0;
        const bool whole = __all_sync(0xffffffffu, lo <= 0 && hi >= C::KT) && !by_pos;
        // (a page of zero scale still gives -inf where masked)
        const float f0 = fmaxf(hdr[0] * fz, 1e-37f), f1 = fmaxf(hdr[1] * fz, 1e-37f);
        const float slot_f = static_cast<float>(slot0 - sv.pos0);
        auto seen = [&](int col) {
          if (by_pos) {
            const int k = kp[col].x;
            return rv.live && slot0 + col < sv.len && (col < hi || k < rv.prefix) && k >= rv.first;
          }
          return col >= lo && col < hi;
        };
        float xs[2][64];
        tmem_ld32(lane_tm, xs[0]);
        tmem_ld32(lane_tm + 32, xs[0] + 32);
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // one page: its scores stay in registers
          const int c0 = half * 64;
          const float f = half ? f1 : f0, lc = hdr[2 + half];
          const float lz = hdr[4 + half];
          float(&x)[64] = xs[half];
          tc::tmem_wait_ld();
          if (MODE == kCap || (MODE == kGeneral && p.cap > 0.0f)) {
            float m4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 64; i += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) m4[k] = tc::max3(m4[k], fabsf(x[i + 2 * k]), fabsf(x[i + 2 * k + 1]));
            const float most = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            if (__all_sync(0xffffffffu, most * f <= kCapSmall * p.cap)) {
              const float fc = f * over, cl = p.cap * kLog2e;
#pragma unroll
              for (int i = 0; i < 64; ++i) x[i] = capped_small(x[i], fc, cl);
            } else {
              // in place in tensor memory, in a loop: the code of 64 values would crowd the loop around it out of the
              // instruction cache (a prompt of documents under a cap of 30 takes 222 us, and 275 with 64 values unrolled
              // here; under a cap of 1, where all come here, 263 and 426)
#pragma unroll 1
              for (int c = c0; c < c0 + 64; c += 16) {
                uint32_t w[16];
                tc::tmem_ld16(lane_tm + c, w);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(capped(__uint_as_float(w[i]) * f, p.cap, over, cap_f));
                tc::tmem_st16(lane_tm + c, w);
              }
              tc::tmem_wait_st();
              tmem_ld32(lane_tm + c0, x);
              tmem_ld32(lane_tm + c0 + 32, x + 32);
              tc::tmem_wait_ld();
            }
          } else if (MODE == kGeneral) {
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i] *= f * kLog2e;
          }
          if (MODE == kGeneral) {
            if (with_pos) {
#pragma unroll
              for (int i = 0; i < 64; ++i) x[i] = fmaf(-rv.slope, fabsf(rv.pos - __int_as_float(kp[c0 + i].y)), x[i]);
            } else {
              const float from = rv.pos - slot_f;
#pragma unroll
              for (int i = 0; i < 64; ++i) x[i] = fmaf(-rv.slope, fabsf(from - static_cast<float>(c0 + i)), x[i]);
            }
          }
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i] = seen(c0 + i) ? x[i] : -INFINITY;
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int i = 4; i < 60; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = tc::max3(mx[k], x[i + 2 * k], x[i + 2 * k + 1]);
          const float m = tc::max3(tc::max3(mx[0], x[60], x[61]), tc::max3(mx[1], x[62], x[63]), fmaxf(mx[2], mx[3]));
          const float tz = MODE == kPlain ? fmaf(m, f, lz) : m + lz, t = tz + lc;
          const bool move = t > R + 8.0f, move_l = tz > L + 8.0f;
          if (__any_sync(0xffffffffu, move || move_l)) {
            const float g = move ? tc::ex2(R - t) : 1.0f;
            if (move) R = t;
            if (move_l) l *= tc::ex2(L - tz), L = tz;
            __syncwarp();
            // what the first page stored (its weights; the output, if that page moved the reference too) is loaded again
            // below: stores and loads of tensor memory have no order of their own
            tc::tmem_wait_st();
            if (half) {  // the first page's weights of this tile
#pragma unroll 1
              for (int c = 0; c < 32; c += 16) {
                uint32_t w[16];
                tc::tmem_ld16(lane_tm + c, w);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float2 v = __half22float2(*reinterpret_cast<__half2*>(&w[i]));
                  w[i] = tc::cvt_half2(v.x * g, v.y * g);
                }
                tc::tmem_st16(lane_tm + c, w);
              }
            }
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
            }
          }
          __syncwarp();  // (tensor memory wants the warp as one)
          // weights are 2^(z + up + 7); no lower than z - L - 53, where they are zero in fp16 and still count in the sum
          const float up = fmaxf(lc - R, (lz - 60.0f) - L), off = up + 7.0f;
          const float from = tc::ex2(fminf(-up - L, 60.0f));  // from the weights' sum to the row's
          uint64_t sum2 = 0;
#pragma unroll
          for (int ch = 0; ch < 64; ch += 32) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const uint64_t y = tc::f2pack(x[ch + i], x[ch + i + 1]);
              const uint64_t z = MODE == kPlain ? tc::fma2(y, tc::f2pack(f, f), tc::f2pack(off, off))
                                                    : tc::add2(y, tc::f2pack(off, off));
              const float p0 = tc::ex2(tc::f2lo(z)), p1 = tc::ex2(tc::f2hi(z));
              sum2 = tc::add2(sum2, tc::f2pack(p0, p1));
              w[i >> 1] = tc::cvt_half2(p0, p1);
            }
            // over columns whose scores this row has read
            tc::tmem_st16(lane_tm + half * 32 + ch / 2, w);
            if (half == 0) tmem_ld32(lane_tm + 64 + ch, xs[1] + ch);  // the next page's, while these are worked on
          }
          l = fmaf(tc::f2lo(sum2) + tc::f2hi(sum2), from, l);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        warp_arrive(&p_full[qt], lane);
      }
    }
  } else if (warp < 12) {
    // =============================================================== unpack K
    set_registers<80>();
    constexpr int RPW = 512 / D, N = 128 / RPW / 4, STEP = 4 * RPW;  // rows per warp load, loads per lane, rows between them
    const int u = tid - 256;
    int r0, g;
    unpack_lane<D>(lane, r0, g);
    r0 += (warp - 8) * RPW;
    const uint32_t to = sbase + C::K0 + unpack_at(r0, g);  // (STEP rows are whole groups of 8: a constant further on)
    const int from = r0 * D + g * 16;
    uint4 x[N];
    int64_t ph[2];
    float ks[2], vs[2];
    int pos = 0;
    float v0 = 0.0f;
    auto load = [&](int j) {
      many_pages(p, sv, b, h, (t0 + j) * 2, ph);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const unsigned char* src = p.c.code[0] + ph[half] * (kPage * D) + from;
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
          x[half * (N / 2) + i] =
              ph[half] < 0 ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4*>(src + i * STEP * D));
      }
      if (u == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ks[i] = ph[i] < 0 ? 0.0f : __ldg(p.c.scale[0] + ph[i]);
          vs[i] = ph[i] < 0 ? -1.0f : __ldg(p.c.scale[1] + ph[i]);
        }
      }
      if (with_pos) pos = ph[u >> 6] < 0 ? 0 : __ldg(p.c.pos + ph[u >> 6] * kPage + (u & 63));
    };
    load(0);
    for (int j = 0; j < T; ++j) {
      if (j >= 2 && !(ok = mbar_wait_warp(&k_empty[j & 1], ((j >> 1) - 1) & 1))) break;
#pragma unroll
      for (int i = 0; i < N; ++i) store_codes<CODE>(x[i], to + (j & 1) * C::TILE + i * STEP * 128);
      // header of the tile; its slot was last read by the softmax of tile j - 4, which tile j - 2's products follow
      float* hdr = reinterpret_cast<float*>(sm + C::HDR0 + (j & 3) * C::HDR);
      if (u == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          hdr[i] = ks[i] * code_unit<CODE>();
          float lc = -INFINITY;  // of zeros, or no such page
          if (vs[i] > 0.0f) {
            if (v0 == 0.0f) *v0_slot = v0 = vs[i];
            const float c = __fdiv_rn(vs[i], v0);
            lc = c > 1e-30f && c < 1e30f ? log2f(c) : log2f(vs[i]) - log2f(v0);
          }
          hdr[2 + i] = lc;
          hdr[4 + i] = vs[i] < 0.0f ? -INFINITY : 0.0f;  // no such page: its keys have no weight
        }
      }
      if (with_pos) reinterpret_cast<int2*>(hdr + 8)[u] = make_int2(pos, __float_as_int(static_cast<float>(pos - sv.pos0)));
      fence_proxy_async_smem();
      warp_arrive(&k_full[j & 1], lane);
      if (lane == 0) mbar_arrive(&h_full[j & 3]);
      if (j + 1 < T) load(j + 1);
    }
  } else {
    if (warp == 15) {
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
    } else {
    // =============================================================== unpack V
    // the three warps take the tile's warp loads (RPW rows each) in turn
    constexpr int RPW = 512 / D, LOADS = 128 / RPW, N = (LOADS + 2) / 3;
    int r0, g;
    unpack_lane<D>(lane, r0, g);
    const int w = warp - 12;
    const int from = r0 * D + g * 16;
    uint4 x[N];
    int64_t ph[2];
    auto load = [&](int j) {
      many_pages(p, sv, b, h, (t0 + j) * 2, ph);
      const unsigned char* src0 = p.c.code[1] + ph[0] * (kPage * D) + from;
      const unsigned char* src1 = p.c.code[1] + (ph[1] - 1) * (kPage * D) + from;  // rows 64 .. 127
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int q = 3 * i + w;  // (warp-uniform)
        const bool late = q >= LOADS / 2;
        x[i] = make_uint4(0, 0, 0, 0);
        if (q < LOADS && ph[late] >= 0) x[i] = __ldg(reinterpret_cast<const uint4*>((late ? src1 : src0) + q * (RPW * D)));
      }
    };
    load(0);
    for (int j = 0; j < T; ++j) {
      if (j >= 2 && !(ok = mbar_wait_warp(&v_empty[j & 1], ((j >> 1) - 1) & 1))) break;
      const uint32_t to = sbase + C::V0 + (j & 1) * C::TILE;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int q = 3 * i + w;
        if (q < LOADS) store_codes<CODE>(x[i], to + unpack_at(q * RPW + r0, g));
      }
      fence_proxy_async_smem();
      warp_arrive(&v_full[j & 1], lane);
      if (j + 1 < T) load(j + 1);
    }
    }
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
    // from the output's reference to the sum's, in two halves: 2^(R - L) may be past float32 where v0 makes up for it
    const float half = tc::ex2(0.5f * (R - L));
    const float inv = part ? half : (l == 0.0f ? 0.0f : __fdiv_rn(half, l)), v0 = *v0_slot * code_unit<CODE>() * half;
    const int64_t pr = (static_cast<int64_t>(split) * p.B * p.c.H + bh) * (static_cast<int64_t>(p.row_tiles) * 256) + row;
    // through the query tile's place in shared memory (its last product is done), to be stored as whole rows
    const uint32_t stage = sbase + C::Q0 + (warp >> 2) * C::TILE + ((tid & 127) >> 3) * 1024 + (tid & 7) * 128;
#pragma unroll 1
    for (int c = 0; ok && c < D; c += 32) {
      __syncwarp();
      float v[32];
      if (T > 0) {
        tmem_ld32(lane_tm + c, v);
        tc::tmem_wait_ld();
      } else {
#pragma unroll
        for (int x = 0; x < 32; ++x) v[x] = 0.0f;
      }
#pragma unroll
      for (int x = 0; x < 32; ++x) v[x] = v[x] * inv * v0;
      if (part) {
        if (rv.live) {
#pragma unroll
          for (int x = 0; x < 32; x += 4)
            *reinterpret_cast<float4*>(p.part_o + pr * D + c + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
        }
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t w[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            w[y] = p.q_bf16 ? tc::cvt_bf162(v[8 * x + 2 * y], v[8 * x + 2 * y + 1]) : tc::cvt_half2(v[8 * x + 2 * y], v[8 * x + 2 * y + 1]);
          const int chunk = c / 8 + x;
          tc::sts128(stage + (chunk >> 3) * (128 * 128) + (((chunk & 7) ^ (tid & 7)) << 4), w[0], w[1], w[2], w[3]);
        }
      }
    }
    __syncwarp();
    if (ok && !part) {
      constexpr int CPR = D / 8, RPI = 32 / CPR;
      const int c = lane % CPR;
      const unsigned char* from = sm + C::Q0 + (warp >> 2) * C::TILE + (c >> 3) * (128 * 128);
      RowWalk at(p, row0 + warp * 32 + lane / CPR, RPI);
      uint16_t* out = p.out + b * p.o_sb + static_cast<int64_t>(h) * p.G * p.o_sh + c * 8;
#pragma unroll 4
      for (int x = 0; x < 32 / RPI; ++x, at.next(p)) {
        const int r = (warp & 3) * 32 + x * RPI + lane / CPR;
        if (at.i < sv.q_len)  // (a row of no query is left as it is)
          *reinterpret_cast<uint4*>(out + at.g * p.o_sh + at.i * p.o_st) =
              lds128(from + (r >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4));
      }
    }
    if (ok && rv.live) {
      if (part)
        p.part_ml[pr] = make_float2(L, l);
      else if (p.lse)
        p.lse[(static_cast<int64_t>(b) * p.Hq + hq) * p.n + i] = l == 0.0f ? -INFINITY : (L - 7.0f + log2f(l)) * kLn2;
    }
    tc::fence_before_sync();
  }
  __syncthreads();
  if (warp == 15) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tm, 512);
  }
}

}  // namespace
}  // namespace vq
