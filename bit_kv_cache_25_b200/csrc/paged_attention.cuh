// Attention over the paged 8-bit cache for few query rows, and the sums of the
// attention weights per cached token.
//
// A row is one (query, query head); the G = Hq / H query heads that share a key
// head are rows of the same problem, row r = i * G + g, so the codes are read
// once for all of them. With z_j = sigma * scale_K * (q . code_j) (capped, biased
// and masked as asked), the output is sum_j e^(z_j - lse) * scale_V * code_j.
//
// Codes are exact in fp16, and so are fp16 queries. A row of bf16 queries is taken
// to fp16 after a power of two that puts its largest magnitude in [2^7, 2^8): exact
// down to 2^-24 of that magnitude, and off by 2^-32 of it at most below (half of
// fp16's smallest step, 2^-25, over 2^7). Products of q . code are exact and sums are
// fp32; a page's scales are factors of its scores and of its share of the output, both
// in fp32. The only other rounding to fewer bits is that of the weights to fp16 before
// the product with V: 2^-11 of each weight at most, where the output's own rounding is
// 2^-8 (bf16) or 2^-11 (fp16) of the sum. Log-sum-exp and sums of weights never see it.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "paged.cuh"
#include "vq_internal.h"

namespace vq {

struct PagedAttnParams {
  PagedPool c;
  const int32_t* lens;
  const int32_t* q_lens;   // or NULL: n
  const int32_t* q_pos;    // or NULL: slot of the query's own token
  const int32_t* prefix;   // or NULL
  const int32_t* first;    // [B][n] or NULL
  const float* slopes;     // [Hq] or NULL
  const uint16_t* q;
  int64_t q_sb, q_sh, q_st;
  uint16_t* out;
  int64_t o_sb, o_sh, o_st;
  float* lse;              // [B][Hq][n]
  int B, Hq, G, n;
  int causal;
  int q_bf16;
  float sigma, cap;        // cap 0: none
  int row_tiles, splits;
  float* part_o;           // [splits][B * H * row_tiles * ROWS][D]
  float2* part_ml;         // same rows: reference (log2 units) and sum
  int accumulate;          // weights kernel: add to what is there
};

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The first product of a sum.
__device__ __forceinline__ void mma_16816_from_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// cap * tanh(z / cap), times log2 e, of z = a * f: its error is a few 2^-24 of the smaller of |z| and the cap, so that a
// large cap is close to none. Two forms:
// |z| <= cap / 4: tanh(x) = x * P(x^2), P of degree 3 interpolated at the Chebyshev nodes of [0, 1/16] (2.5e-09 of itself
// off at most, below float32's own rounding; degree 2 would be 4.0e-07 off, which shows in the weights). Most scores are
// small enough for it, and it takes three multiply-adds where the other takes two turns of the exponential unit: a warp
// decides for all of its values.
constexpr float kCapSmall = 0.25f;
__device__ __forceinline__ float capped_small(float a, float f_over_cap, float cap_log2e) {
  const float x = a * f_over_cap, y = x * x;
  float t = fmaf(-0.05132700516785341f * cap_log2e, y, 0.13323126058764362f * cap_log2e);
  t = fmaf(t, y, -0.33333206285536826f * cap_log2e);
  return x * fmaf(t, y, 0.9999999975205603f * cap_log2e);
}
// Any z, where a warp has larger ones: beyond cap / 4 tanh(x) = 1 - 2 / (e^2x + 1), which saturates without a NaN at both
// ends (and cancels below: its error is a few 2^-24 of the cap).
__device__ __forceinline__ float capped(float z, float cap, float over_cap, float two_log2e_over_cap) {
  const float e = tc::ex2(z * two_log2e_over_cap);
  const float large = (cap - __fdividef(2.0f * cap, e + 1.0f)) * kLog2e;
  return fabsf(z) <= kCapSmall * cap ? capped_small(z, over_cap, cap * kLog2e) : large;
}

// What a row sees: slots [0, hi), or positions below `prefix` up to slot `len`, from position `first` on.
struct RowView {
  int hi;      // one past the last slot that the causal rule (or the length) allows; -1: no such query
  int first;   // lowest position seen
  float pos;   // the query's own position, counted from the call's first query of the sequence
  float slope; // distance bias per position, in log2 units
};

// pos0: position of the first query. Distances are taken between positions counted from it, in float32: exact below
// 2^24, and off by 2^-24 of the distance (and of n) beyond.
struct SeqView {
  int len, q_len, prefix, pos0;
};

__device__ __forceinline__ SeqView seq_view(const PagedAttnParams& p, int b) {
  SeqView s;
  s.len = paged_len(p.c, p.lens, b);
  s.q_len = p.q_lens ? __ldg(p.q_lens + b) : p.n;
  if (s.q_len < 0 || s.q_len > p.n) {
    paged_error();
    s.q_len = s.q_len < 0 ? 0 : p.n;
  }
  s.prefix = p.prefix ? __ldg(p.prefix + b) : 0;
  s.pos0 = p.q_pos ? __ldg(p.q_pos + b) : s.len - s.q_len;
  return s;
}

__device__ __forceinline__ RowView row_view(const PagedAttnParams& p, const SeqView& s, int b, int h, int row) {
  RowView v;
  const int i = row / p.G;
  v.hi = -1;
  v.first = INT32_MAX;
  v.pos = 0.0f;
  v.slope = 0.0f;
  if (i >= s.q_len) return v;
  v.hi = p.causal ? max(0, min(s.len, s.len - s.q_len + i + 1)) : s.len;
  v.first = p.first ? __ldg(p.first + static_cast<int64_t>(b) * p.n + i) : INT32_MIN;
  v.pos = static_cast<float>(i);
  v.slope = p.slopes ? __ldg(p.slopes + h * p.G + row % p.G) * kLog2e : 0.0f;
  return v;
}

// What the scores need beyond the product: nothing but an interval of slots per row; a cap too; or terms that
// depend on positions.
enum PagedMode : int { kPlain = 0, kCap = 1, kGeneral = 2 };

// A row's interval of visible slots, where positions are slots or are not asked for: [lo, hi).
__device__ __forceinline__ void row_interval(const PagedAttnParams& p, const SeqView& s, const RowView& v, bool by_pos,
                                             int& lo, int& hi) {
  lo = by_pos ? 0 : max(v.first, 0);
  hi = max(v.hi, 0);
  if (v.hi >= 0 && p.causal && p.prefix && !by_pos) hi = max(hi, min(s.len, s.prefix));
}

// The B fragments of ROWS query rows (row 8 * half + r for lane 4r + c; the thread's channels are c * D / 4 on).
// Rows past the call's are zero and not read. bf16 rows are multiplied by a power of two that puts their largest
// magnitude in [2^7, 2^8); `back` undoes it, for the rows 8 * half + 2c + e of the thread's scores.
template <int D, int ROWS>
__device__ __forceinline__ void load_q(const PagedAttnParams& p, const SeqView& s, int b, int h, int row0, int lane,
                                       uint32_t (&qb)[D / 16][ROWS / 4], float (&back)[ROWS / 8][2]) {
  constexpr int KS = D / 16;
  const int c = lane & 3;
#pragma unroll
  for (int half = 0; half < ROWS / 8; ++half) {
    const int row = row0 + half * 8 + (lane >> 2);
    const int i = row / p.G, hq = h * p.G + row % p.G;
    uint2 raw[KS];
    const bool live = i < s.q_len;
    const uint16_t* q = p.q + b * p.q_sb + hq * p.q_sh + i * p.q_st + c * (D / 4);
#pragma unroll
    for (int j = 0; j < KS / 2; ++j) {
      const uint4 v = live ? __ldg(reinterpret_cast<const uint4*>(q + j * 8)) : make_uint4(0, 0, 0, 0);
      raw[2 * j] = make_uint2(v.x, v.y);
      raw[2 * j + 1] = make_uint2(v.z, v.w);
    }
    float mine = 1.0f;
    if (p.q_bf16) {
      uint32_t top = 0;  // largest magnitude's bf16 bits
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        top = __vmaxu2(top, raw[k].x & 0x7fff7fffu);
        top = __vmaxu2(top, raw[k].y & 0x7fff7fffu);
      }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = max(min(static_cast<int>(top >> 7) - 127, 119), -119);  // a row of zeros, of tiny values, of infinity
      const float f = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23);
      mine = __uint_as_float(static_cast<uint32_t>(127 - 7 + e) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        raw[k].x = tc::cvt_half2(__uint_as_float(raw[k].x << 16) * f, __uint_as_float(raw[k].x & 0xffff0000u) * f);
        raw[k].y = tc::cvt_half2(__uint_as_float(raw[k].y << 16) * f, __uint_as_float(raw[k].y & 0xffff0000u) * f);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) back[half][e] = __shfl_sync(0xffffffffu, mine, 8 * c + 4 * e);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      qb[k][2 * half] = raw[k].x;      // channels 0, 1 of the thread's four
      qb[k][2 * half + 1] = raw[k].y;  // 2, 3
    }
  }
}

// ---- units: the codes of 32 tokens of a page in shared memory
// Rows of D bytes, their 16-byte chunks permuted so that both the fragment loads of K (two rows of a thread group's
// chunks at a time) and the transposing loads of V (one chunk of eight rows) touch all banks once.
template <int D>
__device__ __forceinline__ uint32_t unit_at(int row, int chunk) {
  return row * D + ((D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4);
}
template <int D>
struct UnitCfg {
  static constexpr int CODES = 32 * D;         // bytes of one tensor's codes
  static constexpr int SCALES = CODES;         // behind K's: K and V scale
  static constexpr int POS = SCALES + 16;      // 32 positions
  static constexpr int K = CODES + 256;
  static constexpr int V = CODES;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros (nothing is read)
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The warp copies half `half` of page slot ph (page * H + h) to `dst`: the codes of one tensor; K's with the scales of
// both, and positions if asked for.
template <int D, int TENSOR>
__device__ __forceinline__ void copy_unit(const PagedPool& c, int64_t ph, int half, uint32_t dst, int lane, bool pos) {
  constexpr int CPR = D / 16, RPI = 32 / CPR;
  const unsigned char* from = c.code[TENSOR] + (ph * kPage + half * 32) * D + lane * 16;
#pragma unroll
  for (int i = 0; i < 32 / RPI; ++i) copy16(dst + unit_at<D>(i * RPI + lane / CPR, lane % CPR), from + i * 512);
  if (TENSOR == 0) {
    if (lane < 2) copy4(dst + UnitCfg<D>::SCALES + lane * 4, (lane ? c.scale[1] : c.scale[0]) + ph);
    if (pos && lane < 8) copy16(dst + UnitCfg<D>::POS + lane * 16, c.pos + ph * kPage + half * 32 + lane * 4);
  }
}

// Raw scores, transposed: s[mt][half][2 * g + e] of lane 4r + c is key 16 * mt + 8 * g + r, row 8 * half + 2c + e.
// (Keys as the products' 16 rows and queries as their 8 columns: no product has rows of nothing, and the fragments of K
// come from the conversions in the registers that the instruction wants.)
template <int D, int CODE, int ROWS>
__device__ __forceinline__ void scores_32(uint32_t unit, const uint32_t (&qb)[D / 16][ROWS / 4], int lane,
                                          float (&s)[2][ROWS / 8][4]) {
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    uint4 k[2][D / 64];
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const uint32_t at = unit + unit_at<D>(mt * 16 + g * 8 + (lane >> 2), (lane & 3) * (D / 64) + j);
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(k[g][j].x), "=r"(k[g][j].y), "=r"(k[g][j].z), "=r"(k[g][j].w) : "r"(at));
      }
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t a[4];
      codes_f16<CODE>((&k[0][ks >> 2].x)[ks & 3], a[0], a[2]);
      codes_f16<CODE>((&k[1][ks >> 2].x)[ks & 3], a[1], a[3]);
#pragma unroll
      for (int half = 0; half < ROWS / 8; ++half) {
        if (ks == 0)
          mma_16816_from_zero(s[mt][half], a, qb[ks][2 * half], qb[ks][2 * half + 1]);
        else
          mma_16816(s[mt][half], a, qb[ks][2 * half], qb[ks][2 * half + 1]);
      }
    }
  }
}

// What the thread's rows 8 * half + 2c + e see.
template <int ROWS>
struct FewRowsView {
  RowView v[ROWS / 8][2];
  int lo[ROWS / 8][2], hi[ROWS / 8][2];
  int hi_max, hi_min, lo_min, lo_max;  // over the tile: bounds of the walk, and of the slots that every row sees

  __device__ __forceinline__ void load(const PagedAttnParams& p, const SeqView& sv, int b, int h, int row0, int lane, bool by_pos) {
    hi_max = 0, hi_min = INT32_MAX, lo_min = INT32_MAX, lo_max = 0;
#pragma unroll
    for (int half = 0; half < ROWS / 8; ++half)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const RowView r = row_view(p, sv, b, h, row0 + half * 8 + 2 * (lane & 3) + e);
        int l, u;
        row_interval(p, sv, r, by_pos, l, u);
        hi_max = max(hi_max, u);
        hi_min = min(hi_min, by_pos ? INT32_MAX : u);
        lo_max = max(lo_max, l);  // (0 where positions decide)
        if (r.hi >= 0) {
          lo_min = min(lo_min, l);
          if (by_pos && p.causal && p.prefix) hi_max = sv.len;
        }
        // with positions every score is masked for itself; the slots here only bound the walk
        v[half][e] = r;
        lo[half][e] = l;
        hi[half][e] = by_pos ? INT32_MAX : u;
      }
    // (unconditional, all four: with the last two in a choice by by_pos, the 16-row kernels for positions and slopes were
    // compiled to ones that masked no slot at all)
    hi_max = __reduce_max_sync(0xffffffffu, hi_max);
    hi_min = __reduce_min_sync(0xffffffffu, hi_min);
    lo_min = __reduce_min_sync(0xffffffffu, lo_min);
    lo_max = __reduce_max_sync(0xffffffffu, lo_max);
  }
};

// Scores to log2 units with cap, bias and masks; -inf where the row does not see the key. pos: the unit's positions, or NULL.
template <int ROWS, int MODE>
__device__ __forceinline__ void finish_scores(const PagedAttnParams& p, const SeqView& sv, const FewRowsView<ROWS>& rows,
                                              float f, const float (&back)[ROWS / 8][2], float cap_f, int slot0, int lane,
                                              const int32_t* pos, float (&s)[2][ROWS / 8][4]) {
  const int prefix = p.causal && p.prefix ? sv.prefix : INT32_MIN;
  const bool masked = slot0 + 32 > rows.hi_min || slot0 < rows.lo_max;  // (warp-uniform)
  const bool by_pos = MODE == kGeneral && pos && (p.first || (p.prefix && p.causal));
  const bool cap = MODE == kCap || (MODE == kGeneral && p.cap > 0.0f);
  float fr[ROWS / 8][2];
#pragma unroll
  for (int half = 0; half < ROWS / 8; ++half)
#pragma unroll
    for (int e = 0; e < 2; ++e) fr[half][e] = f * back[half][e];
#pragma unroll
  for (int x = 0; x < 4; ++x)
#pragma unroll
    for (int half = 0; half < ROWS / 8; ++half)
#pragma unroll
      for (int e = 0; e < 2; ++e) s[x >> 1][half][2 * (x & 1) + e] *= fr[half][e];
  if (cap) {
    float top = 0.0f;
#pragma unroll
    for (int half = 0; half < ROWS / 8; ++half)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(s[0][half][i]), fabsf(s[1][half][i])));
    const float over = 0.5f * kLn2 * cap_f, cl = p.cap * kLog2e;  // (over: 1 / cap)
    if (__all_sync(0xffffffffu, top <= kCapSmall * p.cap)) {
#pragma unroll
      for (int half = 0; half < ROWS / 8; ++half)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[0][half][i] = capped_small(s[0][half][i], over, cl);
          s[1][half][i] = capped_small(s[1][half][i], over, cl);
        }
    } else {
#pragma unroll
      for (int half = 0; half < ROWS / 8; ++half)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[0][half][i] = capped(s[0][half][i], p.cap, over, cap_f);
          s[1][half][i] = capped(s[1][half][i], p.cap, over, cap_f);
        }
    }
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int key = 8 * x + (lane >> 2), slot = slot0 + key;
    int kp = slot;
    float kf = 0.0f;
    if (MODE == kGeneral) {
      if (pos) kp = pos[key];
      kf = static_cast<float>(kp - sv.pos0);
    }
#pragma unroll
    for (int half = 0; half < ROWS / 8; ++half)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const RowView& rv = rows.v[half][e];
        float z = s[x >> 1][half][2 * (x & 1) + e];
        if (MODE == kGeneral) {
          if (!cap) z *= kLog2e;
          z = fmaf(-rv.slope, fabsf(rv.pos - kf), z);
          if (by_pos) {
            const bool see = slot < sv.len && (slot < rv.hi || (kp < prefix && rv.hi >= 0)) && kp >= rv.first;
            z = see ? z : -INFINITY;
          }
        }
        if (masked && (slot < rows.lo[half][e] || slot >= rows.hi[half][e])) z = -INFINITY;
        s[x >> 1][half][2 * (x & 1) + e] = z;
      }
  }
}

// Four channels of one row to the output, and its log-sum-exp. Weights were taken as
// 2^(z - m + 7); a row that saw nothing has sum 0: output 0, log-sum-exp -inf.
template <int D>
__device__ __forceinline__ void write_row(const PagedAttnParams& p, int b, int h, int row, int ch, float4 v, float m,
                                          float l) {
  const int i = row / p.G, hq = h * p.G + row % p.G;
  const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
  uint2 w;
  if (p.q_bf16)
    w = make_uint2(tc::cvt_bf162(v.x * inv, v.y * inv), tc::cvt_bf162(v.z * inv, v.w * inv));
  else
    w = make_uint2(tc::cvt_half2(v.x * inv, v.y * inv), tc::cvt_half2(v.z * inv, v.w * inv));
  *reinterpret_cast<uint2*>(p.out + b * p.o_sb + hq * p.o_sh + i * p.o_st + ch) = w;
  if (ch == 0 && p.lse)
    p.lse[(static_cast<int64_t>(b) * p.Hq + hq) * p.n + i] = l == 0.0f ? -INFINITY : (m - 7.0f + log2f(l)) * kLn2;
}

constexpr int kFewWarps = 4;
constexpr int kFewWarpsAlone = 12;  // where one CTA takes all pages of a short sequence

template <int D, int ROWS, int WARPS>
struct FewCfg {
  static constexpr int RING = WARPS * (UnitCfg<D>::K + UnitCfg<D>::V);
  static constexpr int JOIN = WARPS * ROWS * (D + 2) * 4;  // afterwards, over the units
  static constexpr int SMEM = RING > JOIN ? RING : JOIN;
};

// Few rows: one CTA of 4 (or 12) warps per (split of the pages, 16- or 8-row tile, key head,
// sequence). Every warp walks 32-token units of codes on its own. Its own asynchronous
// copies bring the next unit's K as soon as this one's scores are taken, and the next V as
// soon as this one's products are: one buffer each, so that 16 warps fit an SM. What limits
// is the warps' own chain of loads, conversions and products (766 instructions a unit,
// 0.53 issued a cycle and scheduler), so warps count for more than bytes in flight:
// 32 ragged sequences of up to 10521 tokens, 8 key heads, took 126 us with three units in
// flight and 8 warps an SM, 107 with one and 16, 96 with the scores transposed, and 90 us
// (4.8 TB/s) with more splits.
// K codes are read as the fragments of Q K^T, channels paired off between Q and K as one
// wide load brings them; V codes by transposing 16-bit loads, which bring a thread two
// channels of two tokens, the fragments of V^T P^T.
template <int D, int CODE, int ROWS, int MODE, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) paged_few_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int KS = D / 16;
  constexpr int MT = D / 16;  // 16-channel tiles of the output
  constexpr int NH = ROWS / 8;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = lane & 3, r = lane >> 2;
  // row tiles of one (sequence, head, split) are neighbours: they share its codes in L2
  const int tile = blockIdx.x % p.row_tiles;
  const int split = (blockIdx.x / p.row_tiles) % p.splits;
  const int bh = blockIdx.x / (p.row_tiles * p.splits);
  const int b = bh / p.c.H, h = bh - b * p.c.H;
  const int row0 = tile * ROWS;
  const bool with_pos = MODE == kGeneral && p.c.pos;
  const bool by_pos = with_pos && (p.first || (p.prefix && p.causal));  // positions decide what is seen

  const SeqView sv = seq_view(p, b);
  FewRowsView<ROWS> view;
  view.load(p, sv, b, h, row0, lane, by_pos);
  const int pg_lo = min(view.lo_min, view.hi_max) / kPage, pg_hi = (view.hi_max + kPage - 1) / kPage;
  const int per = (pg_hi - pg_lo + p.splits - 1) / p.splits;
  const int pg0 = pg_lo + split * per, pg1 = min(pg_hi, pg0 + per);
  const int units = max(0, pg1 - pg0) * 2;

  // the warp's two buffers; page ids one unit further ahead than the copies
  unsigned char* mine = smem_raw + warp * (UnitCfg<D>::K + UnitCfg<D>::V);
  const uint32_t k_at = smem_addr(mine), v_at = k_at + UnitCfg<D>::K;
  const float* head = reinterpret_cast<const float*>(mine + UnitCfg<D>::SCALES);
  auto page_of = [&](int u) -> int64_t {  // page * H + h of a unit, -1: none
    const int page = u < units ? paged_page(p.c, b, pg0 + u / 2) : -1;
    return page < 0 ? -1 : static_cast<int64_t>(page) * p.c.H + h;
  };
  int64_t ph = page_of(warp), ph_next = page_of(warp + WARPS);
  if (ph >= 0) copy_unit<D, 0>(p.c, ph, warp & 1, k_at, lane, with_pos);
  copy_commit();
  if (ph >= 0) copy_unit<D, 1>(p.c, ph, warp & 1, v_at, lane, false);
  copy_commit();

  uint32_t qb[KS][ROWS / 4];
  float back[NH][2];
  load_q<D, ROWS>(p, sv, b, h, row0, lane, qb, back);
  const float qk = p.sigma * code_unit<CODE>() * (MODE == kPlain ? kLog2e : 1.0f);
  const float cap_f = MODE != kPlain && p.cap > 0.0f ? 2.0f * kLog2e / p.cap : 0.0f;

  // output of rows 8 * half + 2c + e (second index 2 * half + e): channels 16 * mt + 2 * r (o) and one above (od)
  float o[MT][2 * NH], od[MT][2 * NH];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int e = 0; e < 2 * NH; ++e) o[mt][e] = od[mt][e] = 0.0f;
  // reference (the same on the eight lanes of a row) and sum (each lane its keys')
  float ref[NH][2], sum[NH][2];
#pragma unroll
  for (int half = 0; half < NH; ++half)
#pragma unroll
    for (int e = 0; e < 2; ++e) ref[half][e] = -INFINITY, sum[half][e] = 0.0f;

  for (int u = warp; u < units; u += WARPS) {
    const bool there = ph >= 0;  // (warp-uniform) tokens of a page out of range count as unseen
    ph = ph_next;
    ph_next = page_of(u + 2 * WARPS);
    copy_wait<1>();
    __syncwarp();  // K is there for every lane
    float s[2][NH][4];
    const float ks = head[0], vs = head[1] * code_unit<CODE>();
    if (there) {
      scores_32<D, CODE, ROWS>(k_at, qb, lane, s);
      finish_scores<ROWS, MODE>(p, sv, view, ks * qk, back, cap_f, (pg0 + u / 2) * kPage + (u & 1) * 32, lane,
                                with_pos ? reinterpret_cast<const int32_t*>(head + 4) : nullptr, s);
    }
    __syncwarp();  // every lane has left K
    if (ph >= 0) copy_unit<D, 0>(p.c, ph, u & 1, k_at, lane, with_pos);  // (units of a warp are all first or all second halves)
    copy_commit();
    __syncwarp();  // (some lanes copied the scales: the matrix instructions below want the warp as one)
    if (!there) {
      if (ph >= 0) copy_unit<D, 1>(p.c, ph, u & 1, v_at, lane, false);
      copy_commit();
      continue;
    }
    // a row's reference only moves when a score passes it by 8 (weights up to 2^15): mostly one vote
    float top[NH][2];
    bool move = false;
#pragma unroll
    for (int half = 0; half < NH; ++half)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[half][e] = fmaxf(fmaxf(s[0][half][e], s[0][half][2 + e]), fmaxf(s[1][half][e], s[1][half][2 + e]));
        move |= top[half][e] > ref[half][e] + 8.0f;
      }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int half = 0; half < NH; ++half) {
        float g[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m = top[half][e];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
          const float to = m > ref[half][e] + 8.0f ? m : ref[half][e];
          g[e] = to == ref[half][e] ? 1.0f : tc::ex2(ref[half][e] - to);
          ref[half][e] = to;
          sum[half][e] *= g[e];
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            o[mt][2 * half + e] *= g[e];
            od[mt][2 * half + e] *= g[e];
          }
      }
    }
    uint32_t pb[NH][4];  // weights as B fragments: keys 8x + 2c, + 1 of row 8 * half + r
#pragma unroll
    for (int half = 0; half < NH; ++half) {
      const float base0 = (ref[half][0] == -INFINITY ? 0.0f : ref[half][0]) - 7.0f;
      const float base1 = (ref[half][1] == -INFINITY ? 0.0f : ref[half][1]) - 7.0f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float p0 = tc::ex2(s[x >> 1][half][2 * (x & 1)] - base0), p1 = tc::ex2(s[x >> 1][half][2 * (x & 1) + 1] - base1);
        sum[half][0] += p0;
        sum[half][1] += p1;
        const uint32_t w = tc::cvt_half2(p0, p1);  // key 8x + r, rows 2c, 2c + 1
        asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pb[half][x]) : "r"(w));
      }
    }
    copy_wait<1>();
    __syncwarp();  // V is there for every lane
    // eight keys by one 16-byte chunk of channels per matrix: the lane's register has channels 2r, 2r + 1 of keys 2c, 2c + 1
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t v[4];  // keys 0-7, 8-15, 16-23, 24-31
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                   : "r"(v_at + unit_at<D>(lane, mt)));
      float acc[NH][4];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t a[4];
        codes_f16_of_two<CODE>(v[2 * kk], a[0], a[1]);
        codes_f16_of_two<CODE>(v[2 * kk + 1], a[2], a[3]);
#pragma unroll
        for (int half = 0; half < NH; ++half) {
          if (kk == 0)
            mma_16816_from_zero(acc[half], a, pb[half][0], pb[half][1]);
          else
            mma_16816(acc[half], a, pb[half][2], pb[half][3]);
        }
      }
#pragma unroll
      for (int half = 0; half < NH; ++half) {
        o[mt][2 * half] = fmaf(vs, acc[half][0], o[mt][2 * half]);
        o[mt][2 * half + 1] = fmaf(vs, acc[half][1], o[mt][2 * half + 1]);
        od[mt][2 * half] = fmaf(vs, acc[half][2], od[mt][2 * half]);
        od[mt][2 * half + 1] = fmaf(vs, acc[half][3], od[mt][2 * half + 1]);
      }
    }
    __syncwarp();  // every lane has left V
    if (ph >= 0) copy_unit<D, 1>(p.c, ph, u & 1, v_at, lane, false);
    copy_commit();
  }

  // join the warps, over the units
  copy_wait<0>();
  __syncthreads();
  float* sm_o = reinterpret_cast<float*>(smem_raw);  // [warp][row][D]
  float* sm_ref = sm_o + WARPS * ROWS * D;       // [warp][row]
  float* sm_sum = sm_ref + WARPS * ROWS;
#pragma unroll
  for (int half = 0; half < NH; ++half) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = sum[half][e];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
      if (r == 0) {
        sm_ref[warp * ROWS + half * 8 + 2 * c + e] = ref[half][e];
        sm_sum[warp * ROWS + half * 8 + 2 * c + e] = l;
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float* at = sm_o + (warp * ROWS + half * 8 + 2 * c) * D + mt * 16 + 2 * r;
      *reinterpret_cast<float2*>(at) = make_float2(o[mt][2 * half], od[mt][2 * half]);
      *reinterpret_cast<float2*>(at + D) = make_float2(o[mt][2 * half + 1], od[mt][2 * half + 1]);
    }
  }
  __syncthreads();
  for (int x = tid; x < ROWS * D / 4; x += WARPS * 32) {
    const int row = x / (D / 4), ch = (x % (D / 4)) * 4;
    const int i = (row0 + row) / p.G;
    if (i >= sv.q_len) continue;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) m = fmaxf(m, sm_ref[w * ROWS + row]);
    float l = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float m_w = sm_ref[w * ROWS + row];
      const float g = m_w == m ? 1.0f : tc::ex2(m_w - m);  // (a NaN's sum goes on)
      l += g * sm_sum[w * ROWS + row];
      const float4 a = *reinterpret_cast<const float4*>(sm_o + (w * ROWS + row) * D + ch);
      v.x = fmaf(g, a.x, v.x), v.y = fmaf(g, a.y, v.y), v.z = fmaf(g, a.z, v.z), v.w = fmaf(g, a.w, v.w);
    }
    if (p.splits > 1) {
      const int64_t pr = (static_cast<int64_t>(split) * p.B * p.c.H + bh) * (static_cast<int64_t>(p.row_tiles) * ROWS) + row0 + row;
      *reinterpret_cast<float4*>(p.part_o + pr * D + ch) = v;
      if (ch == 0) p.part_ml[pr] = make_float2(m, l);
    } else {
      write_row<D>(p, b, h, row0 + row, ch, v, m, l);
    }
  }
}

// Joins the splits: one CTA per row, whose WARPS warps take the splits in turn (a warp alone would wait for one split
// after the other: 148 of them took 60 us) and meet in shared memory, always in the same order.
template <int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) paged_join_kernel(const __grid_constant__ PagedAttnParams p, int rows_pad) {
  constexpr int C = D / 32;  // channels per lane
  __shared__ float sm_ref[WARPS], sm_sum[WARPS];
  __shared__ float sm_o[WARPS][D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = p.n * p.G;
  const int bh = blockIdx.x / rows, row = blockIdx.x % rows;
  const int b = bh / p.c.H, h = bh % p.c.H;
  const SeqView sv = seq_view(p, b);
  if (row / p.G >= sv.q_len) return;
  const int64_t stride = static_cast<int64_t>(p.B) * p.c.H * rows_pad;
  const int64_t at = static_cast<int64_t>(bh) * rows_pad + row;
  float m = -INFINITY, l = 0.0f;
  for (int s = warp + WARPS * lane; s < p.splits; s += WARPS * 32) m = fmaxf(m, __ldg(&p.part_ml[at + s * stride].x));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float v[C];
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] = 0.0f;
#pragma unroll 8
  for (int s = warp; s < p.splits; s += WARPS) {
    const float2 ml = __ldg(&p.part_ml[at + s * stride]);
    const float* o = p.part_o + (at + s * stride) * D + lane * C;
    const float g = ml.x == m ? 1.0f : tc::ex2(ml.x - m);  // (a NaN's sum goes on)
    l = fmaf(g, ml.y, l);
    if constexpr (C == 4) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(o));
      v[0] = fmaf(g, a.x, v[0]), v[1] = fmaf(g, a.y, v[1]), v[2] = fmaf(g, a.z, v[2]), v[3] = fmaf(g, a.w, v[3]);
    } else {
      const float2 a = __ldg(reinterpret_cast<const float2*>(o));
      v[0] = fmaf(g, a.x, v[0]), v[1] = fmaf(g, a.y, v[1]);
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i) sm_o[warp][lane * C + i] = v[i];
  if (lane == 0) sm_ref[warp] = m, sm_sum[warp] = l;
  __syncthreads();
  if (tid >= D / 4) return;
  m = sm_ref[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) m = fmaxf(m, sm_ref[w]);
  l = 0.0f;
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const float g = sm_ref[w] == m ? 1.0f : tc::ex2(sm_ref[w] - m);
    l = fmaf(g, sm_sum[w], l);
    const float4 a = *reinterpret_cast<const float4*>(&sm_o[w][tid * 4]);
    x.x = fmaf(g, a.x, x.x), x.y = fmaf(g, a.y, x.y), x.z = fmaf(g, a.z, x.z), x.w = fmaf(g, a.w, x.w);
  }
  write_row<D>(p, b, h, row, tid * 4, x, m, l);
}

constexpr int kSumStages = 3;  // K units in a warp's ring: one worked on, two on their way

// Sums of the attention weights, few rows: every warp walks 32-token units of K as above, the query rows as fragments
// in registers. A token's weights are summed over the rows of a tile by shuffles in a fixed order, and tile by tile by
// one warp: results repeat to the bit. Bound by memory: the K codes, once per row tile.
template <int D, int CODE, int ROWS, int MODE>
__global__ void __launch_bounds__(kFewWarps * 32) paged_weights_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int KS = D / 16, NH = ROWS / 8;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = lane & 3, r = lane >> 2;
  const int split = blockIdx.x % p.splits;
  const int bh = blockIdx.x / p.splits;
  const int b = bh / p.c.H, h = bh - b * p.c.H;
  const bool with_pos = MODE == kGeneral && p.c.pos;
  const bool by_pos = with_pos && (p.first || (p.prefix && p.causal));  // positions decide what is seen
  const SeqView sv = seq_view(p, b);
  const int pages = (sv.len + kPage - 1) / kPage;
  const int per = (pages + p.splits - 1) / p.splits;
  const int pg0 = split * per, pg1 = min(pages, pg0 + per);
  const int units = max(0, pg1 - pg0) * 2;
  const int rows = sv.q_len * p.G;

  unsigned char* ring_at = smem_raw + warp * (kSumStages * UnitCfg<D>::K);
  const uint32_t ring = smem_addr(ring_at);
  const float qk = p.sigma * code_unit<CODE>() * (MODE == kPlain ? kLog2e : 1.0f);
  const float cap_f = MODE != kPlain && p.cap > 0.0f ? 2.0f * kLog2e / p.cap : 0.0f;
  auto page_of = [&](int u) -> int64_t {  // page * H + h of a unit, -1: none
    const int page = u < units ? paged_page(p.c, b, pg0 + u / 2) : -1;
    return page < 0 ? -1 : static_cast<int64_t>(page) * p.c.H + h;
  };
  int row0 = 0;
  do {  // (once where the rows fit a tile)
    int64_t ph[kSumStages];  // of this unit and those on their way
#pragma unroll
    for (int i = 0; i < kSumStages; ++i) ph[i] = page_of(warp + i * kFewWarps);
#pragma unroll
    for (int i = 0; i < kSumStages - 1; ++i) {
      if (ph[i] >= 0) copy_unit<D, 0>(p.c, ph[i], warp & 1, ring + i * UnitCfg<D>::K, lane, with_pos);
      copy_commit();
    }
    FewRowsView<ROWS> view;
    view.load(p, sv, b, h, row0, lane, by_pos);
    uint32_t qb[KS][ROWS / 4];
    float back[NH][2], base[NH][2];
    load_q<D, ROWS>(p, sv, b, h, row0, lane, qb, back);
#pragma unroll
    for (int half = 0; half < NH; ++half)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = row0 + half * 8 + 2 * c + e;
        base[half][e] = INFINITY;  // no such row, or one that saw nothing
        if (view.v[half][e].hi >= 0) {
          const float lse = __ldg(p.lse + (static_cast<int64_t>(b) * p.Hq + h * p.G + row % p.G) * p.n + row / p.G);
          if (lse != -INFINITY) base[half][e] = lse * kLog2e;
        }
      }
    int stage = 0;
    for (int u = warp; u < units; u += kFewWarps) {
      copy_wait<kSumStages - 2>();
      __syncwarp();  // this unit is there for every lane, and every lane has left the stage that is filled next
      if (ph[kSumStages - 1] >= 0)
        copy_unit<D, 0>(p.c, ph[kSumStages - 1], u & 1, ring + (stage == 0 ? kSumStages - 1 : stage - 1) * UnitCfg<D>::K, lane, with_pos);
      copy_commit();
      __syncwarp();  // (some lanes copied the scales: the matrix instructions below want the warp as one)
      const int64_t at_page = ph[0];
#pragma unroll
      for (int i = 0; i < kSumStages - 1; ++i) ph[i] = ph[i + 1];
      ph[kSumStages - 1] = page_of(u + kSumStages * kFewWarps);
      const uint32_t unit = ring + stage * UnitCfg<D>::K;
      const float* head = reinterpret_cast<const float*>(ring_at + stage * UnitCfg<D>::K + UnitCfg<D>::SCALES);
      if (++stage == kSumStages) stage = 0;
      if (at_page < 0) continue;
      const int32_t* pos = with_pos ? reinterpret_cast<const int32_t*>(head + 4) : nullptr;
      const int slot0 = (pg0 + u / 2) * kPage + (u & 1) * 32;
      float s[2][NH][4];
      scores_32<D, CODE, ROWS>(unit, qb, lane, s);
      finish_scores<ROWS, MODE>(p, sv, view, head[0] * qk, back, cap_f, slot0, lane, pos, s);
      float mine = 0.0f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {  // key 8x + r: over the thread's rows, then over the four threads of the key
        float w = 0.0f;
#pragma unroll
        for (int half = 0; half < NH; ++half)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float z = s[x >> 1][half][2 * (x & 1) + e];  // (an unseen key has no weight whatever the row's lse, NaN included)
            w += base[half][e] == INFINITY || z == -INFINITY ? 0.0f : tc::ex2(z - base[half][e]);
          }
        w += __shfl_xor_sync(0xffffffffu, w, 1);
        w += __shfl_xor_sync(0xffffffffu, w, 2);
        if (x == c) mine = w;
      }
      const int key = 8 * c + r;
      if (slot0 + key < sv.len) {
        float* at = p.c.weight + at_page * kPage + (u & 1) * 32 + key;
        *at = p.accumulate || row0 > 0 ? *at + mine : mine;
      }
    }
    copy_wait<0>();
    __syncwarp();
    row0 += ROWS;
  } while (row0 < rows);
}

}  // namespace
}  // namespace vq
