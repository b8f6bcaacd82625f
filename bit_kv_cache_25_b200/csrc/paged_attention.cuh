// Attention over the paged 8-bit cache for few query rows, and the sums of the
// attention weights per cached token.
//
// A row is one (query, query head); the G = Hq / H query heads that share a key
// head are rows of the same problem, row r = i * G + g, so the codes are read
// once for all of them. With z_j = sigma * scale_K * (q . code_j) (capped, biased
// and masked as asked), the output is sum_j e^(z_j - lse) * scale_V * code_j.
//
// Codes are exact in fp16 and so are the queries after a power of two per row,
// so the products of q . code are exact and sums are fp32; a page's scales are
// factors of its scores and of its share of the output, both in fp32. The only
// rounding to fewer bits is that of the weights to fp16 before the product with
// V: 2^-12 of each weight, where the output's own rounding is 2^-9 (bf16) or
// 2^-12 (fp16) of the sum. Log-sum-exp and sums of weights never see it.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "paged.cuh"

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

// cap * tanh(z / cap), times log2 e. tanh(x) = 1 - 2 / (e^2x + 1): its error is a few
// 2^-24 of the cap, and it saturates without a NaN at both ends.
__device__ __forceinline__ float capped(float z, float cap, float two_log2e_over_cap) {
  const float e = tc::ex2(z * two_log2e_over_cap);
  return (cap - __fdividef(2.0f * cap, e + 1.0f)) * kLog2e;
}

// What a row sees: slots [0, hi), or positions below `prefix` up to slot `len`, from position `first` on.
struct RowView {
  int hi;      // one past the last slot that the causal rule (or the length) allows; -1: no such query
  int first;   // lowest position seen
  int pos;     // the query's own position
  float slope; // distance bias per position, in log2 units
};

struct SeqView {
  int len, q_len, prefix;
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
  return s;
}

__device__ __forceinline__ RowView row_view(const PagedAttnParams& p, const SeqView& s, int b, int h, int row) {
  RowView v;
  const int i = row / p.G;
  v.hi = -1;
  v.first = INT32_MAX;
  v.pos = 0;
  v.slope = 0.0f;
  if (i >= s.q_len) return v;
  v.hi = p.causal ? max(0, min(s.len, s.len - s.q_len + i + 1)) : s.len;
  v.first = p.first ? __ldg(p.first + static_cast<int64_t>(b) * p.n + i) : INT32_MIN;
  v.pos = p.q_pos ? __ldg(p.q_pos + b) + i : s.len - s.q_len + i;
  v.slope = p.slopes ? __ldg(p.slopes + h * p.G + row % p.G) * kLog2e : 0.0f;
  return v;
}

// The A fragments of 16 query rows (rows r and r + 8 of lane 4r + c): channel order
// as in the K loads below. Rows past the call's are zero and not read. bf16 rows are
// multiplied by a power of two that puts their largest magnitude in [2^7, 2^8); `back`
// undoes it.
template <int D, int ROWS>
__device__ __forceinline__ void load_q(const PagedAttnParams& p, const SeqView& s, int b, int h, int row0, int lane,
                                       uint32_t (&qa)[D / 16][ROWS / 4], float (&back)[ROWS / 8]) {
  constexpr int KS = D / 16;
  const int c = lane & 3;
#pragma unroll
  for (int half = 0; half < ROWS / 8; ++half) {
    const int row = row0 + half * 8 + (lane >> 2);
    const int i = row / p.G, hq = h * p.G + row % p.G;
    uint2 raw[KS];
    const bool live = i < s.q_len;
    const uint16_t* q = p.q + b * p.q_sb + hq * p.q_sh + i * p.q_st;
#pragma unroll
    for (int j = 0; j < KS / 4; ++j) {
      uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
      if (live) {
        v0 = __ldg(reinterpret_cast<const uint4*>(q + j * 64 + c * 16));
        v1 = __ldg(reinterpret_cast<const uint4*>(q + j * 64 + c * 16 + 8));
      }
      raw[4 * j] = make_uint2(v0.x, v0.y);
      raw[4 * j + 1] = make_uint2(v0.z, v0.w);
      raw[4 * j + 2] = make_uint2(v1.x, v1.y);
      raw[4 * j + 3] = make_uint2(v1.z, v1.w);
    }
    back[half] = 1.0f;
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
      back[half] = __uint_as_float(static_cast<uint32_t>(127 - 7 + e) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        raw[k].x = tc::cvt_half2(__uint_as_float(raw[k].x << 16) * f, __uint_as_float(raw[k].x & 0xffff0000u) * f);
        raw[k].y = tc::cvt_half2(__uint_as_float(raw[k].y << 16) * f, __uint_as_float(raw[k].y & 0xffff0000u) * f);
      }
    }
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      // a0: rows r, channels 0,1 of the thread's four; a1: rows r + 8; a2, a3: channels 2,3
      qa[k][half] = raw[k].x;
      qa[k][ROWS / 8 + half] = raw[k].y;
    }
  }
}

template <int ROWS>
__device__ __forceinline__ void mma_rows(float (&d)[4], const uint32_t (&qa)[ROWS / 4], uint32_t b0, uint32_t b1) {
  if (ROWS == 16) {
    const uint32_t a[4] = {qa[0], qa[1], qa[2 % (ROWS / 4)], qa[3 % (ROWS / 4)]};
    mma_16816(d, a, b0, b1);
  } else {
    const uint32_t a[4] = {qa[0], 0u, qa[1], 0u};
    mma_16816(d, a, b0, b1);
  }
}

// K codes of 32 keys of a page, for lane 4r + c: key 8 * nt + r, 16 channels at 64 * j + 16 * c.
template <int D>
__device__ __forceinline__ void load_k(const unsigned char* k, int lane, uint4 (&kr)[4][D / 64]) {
#pragma unroll
  for (int nt = 0; nt < 4; ++nt)
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
      kr[nt][j] = __ldg(reinterpret_cast<const uint4*>(k + (nt * 8 + (lane >> 2)) * D + j * 64 + (lane & 3) * 16));
}

// Raw scores of ROWS rows and 32 keys.
template <int D, int CODE, int ROWS>
__device__ __forceinline__ void scores_32(const uint4 (&kr)[4][D / 64], const uint32_t (&qa)[D / 16][ROWS / 4],
                                          float (&s)[4][4]) {
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t b0, b1;
      codes_f16<CODE>((&kr[nt][ks >> 2].x)[ks & 3], b0, b1);
      mma_rows<ROWS>(s[nt], qa[ks], b0, b1);
    }
  }
}

// Scores to log2 units with cap, bias and masks; -inf where the row does not see the key.
// s[nt][2 * half + e]: row half, key slot0 + 8 * nt + 2 * c + e.
template <int ROWS, bool BIAS>
__device__ __forceinline__ void finish_scores(const PagedAttnParams& p, const SeqView& sv, const RowView (&rv)[ROWS / 8],
                                              const float (&f)[ROWS / 8], float cap_f, int slot0, int lane, bool masked,
                                              const int32_t* pos, float (&s)[4][4]) {
#pragma unroll
  for (int nt = 0; nt < 4; ++nt)
#pragma unroll
    for (int half = 0; half < ROWS / 8; ++half)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float z = s[nt][2 * half + e];
        const int key = nt * 8 + 2 * (lane & 3) + e;
        const int slot = slot0 + key;
        if (BIAS) {
          z *= f[half];  // natural units
          z = p.cap > 0.0f ? capped(z, p.cap, cap_f) : z * kLog2e;
          const int kp = pos ? __ldg(pos + key) : slot;
          z = fmaf(-rv[half].slope, fabsf(static_cast<float>(rv[half].pos - kp)), z);
          const bool see = slot < sv.len && (slot < rv[half].hi || (kp < sv.prefix && rv[half].hi >= 0)) && kp >= rv[half].first;
          z = see ? z : -INFINITY;
        } else {
          z *= f[half];  // log2 units
          if (masked && slot >= rv[half].hi) z = -INFINITY;
        }
        s[nt][2 * half + e] = z;
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

// Few rows: one CTA of four warps per (split of the pages, 16- or 8-row tile, key head,
// sequence). Every warp walks 32-key units on its own with codes loaded straight into the
// MMA fragments: channels are paired off between Q and K, and keys between the weights and
// V, so that a thread's fragment is what one wide load brings it, and no shared memory is
// used until the warps' results are joined. K of the next unit is loaded while this one's
// weights are computed, V of it while the next scores are. Bound by memory: the units'
// codes, once.
template <int D, int CODE, int ROWS, bool BIAS>
__global__ void __launch_bounds__(kFewWarps * 32) paged_few_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int KS = D / 16;
  constexpr int MT = D / 16;  // 16-channel tiles of the output
  constexpr int NH = ROWS / 8;
  __shared__ float sm_o[kFewWarps][ROWS][D];
  __shared__ float sm_ref[kFewWarps][ROWS], sm_sum[kFewWarps][ROWS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = lane & 3, r = lane >> 2;
  // row tiles of one (sequence, head, split) are neighbours: they share its codes in L2
  const int tile = blockIdx.x % p.row_tiles;
  const int split = (blockIdx.x / p.row_tiles) % p.splits;
  const int bh = blockIdx.x / (p.row_tiles * p.splits);
  const int b = bh / p.c.H, h = bh - b * p.c.H;
  const int row0 = tile * ROWS;

  const SeqView sv = seq_view(p, b);
  RowView rv[NH];
  int hi_max = -1, hi_min = INT32_MAX, first_min = INT32_MAX;
#pragma unroll
  for (int half = 0; half < NH; ++half) {
    rv[half] = row_view(p, sv, b, h, row0 + half * 8 + r);
    hi_max = max(hi_max, rv[half].hi);
    hi_min = min(hi_min, rv[half].hi);
    first_min = min(first_min, rv[half].first);
  }
  hi_max = __reduce_max_sync(0xffffffffu, hi_max);
  hi_min = __reduce_min_sync(0xffffffffu, hi_min);
  first_min = __reduce_min_sync(0xffffffffu, first_min);
  // pages that any row can see
  if (BIAS && hi_max >= 0 && p.prefix) hi_max = max(hi_max, p.c.pos ? sv.len : min(sv.len, sv.prefix));
  int pg_lo = 0;
  if (BIAS && p.first && !p.c.pos) pg_lo = max(0, min(first_min, hi_max)) / kPage;
  const int pg_hi = (max(hi_max, 0) + kPage - 1) / kPage;
  const int per = (max(0, pg_hi - pg_lo) + p.splits - 1) / p.splits;
  const int pg0 = pg_lo + split * per, pg1 = min(pg_hi, pg0 + per);
  const int units = max(0, pg1 - pg0) * 2;

  uint32_t qa[KS][ROWS / 4];
  float back[NH];
  load_q<D, ROWS>(p, sv, b, h, row0, lane, qa, back);
  const float qk = p.sigma * code_unit<CODE>() * (BIAS ? 1.0f : kLog2e);
  const float cap_f = BIAS && p.cap > 0.0f ? 2.0f * kLog2e / p.cap : 0.0f;

  // output of rows 8 * half + 2c + e (second index 2 * half + e): channels r * D / 8 + 2 * mt (o) and one above (od)
  float o[MT][2 * NH], od[MT][2 * NH];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int e = 0; e < 2 * NH; ++e) o[mt][e] = od[mt][e] = 0.0f;
  float ref[NH], sum[NH];
#pragma unroll
  for (int half = 0; half < NH; ++half) ref[half] = -INFINITY, sum[half] = 0.0f;

  uint4 kr[4][D / 64];
  // V codes of 32 keys: for k-step kk, keys 16kk + {2c, 2c+1, 2c+8, 2c+9}, D / 8 channels at r * D / 8
  uint32_t vr[2][4][D / 32];
  float ks_next = 0.0f, vs_next = 0.0f;
  const unsigned char* kbase = nullptr;
  const unsigned char* vbase = nullptr;
  const int32_t* pos_next = nullptr;
  bool ok_next = false;
  auto locate = [&](int u) {
    const int page = paged_page(p.c, b, pg0 + u / 2);
    ok_next = page >= 0;
    const int64_t ph = static_cast<int64_t>(max(page, 0)) * p.c.H + h;  // a bad page's codes are read from page 0 and masked
    ks_next = __ldg(p.c.scale[0] + ph);
    vs_next = ok_next ? __ldg(p.c.scale[1] + ph) : 0.0f;
    const int64_t at = (ph * kPage + (u & 1) * 32) * D;
    kbase = p.c.code[0] + at;
    vbase = p.c.code[1] + at;
    pos_next = p.c.pos ? p.c.pos + ph * kPage + (u & 1) * 32 : nullptr;
  };
  auto load_v = [&]() {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const unsigned char* v = vbase + (kk * 16 + 2 * c + (x & 1) + (x >> 1) * 8) * D + r * (D / 8);
        if constexpr (D == 128) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(v));
          vr[kk][x][0] = w.x, vr[kk][x][1] = w.y, vr[kk][x][2] = w.z, vr[kk][x][3] = w.w;
        } else {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(v));
          vr[kk][x][0] = w.x, vr[kk][x][1] = w.y;
        }
      }
  };
  if (warp < units) {
    locate(warp);
    load_k<D>(kbase, lane, kr);
    load_v();
  }
  for (int u = warp; u < units; u += kFewWarps) {
    const float ks = ks_next, vs = vs_next;
    const bool ok = ok_next;
    const int32_t* pos = pos_next;
    const int slot0 = (pg0 + u / 2) * kPage + (u & 1) * 32;
    float s[4][4];
    scores_32<D, CODE, ROWS>(kr, qa, s);
    const bool more = u + kFewWarps < units;
    if (more) {
      locate(u + kFewWarps);
      load_k<D>(kbase, lane, kr);
    }
    float f[NH];
#pragma unroll
    for (int half = 0; half < NH; ++half) f[half] = ks * qk * back[half];
    const bool masked = !ok || slot0 + 32 > hi_min;
    finish_scores<ROWS, BIAS>(p, sv, rv, f, cap_f, slot0, lane, masked, pos, s);
    if (!ok) {
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = -INFINITY;
    }
    // a row's reference only moves when its maximum passes it by 8 (weights up to 2^15)
    float top[NH];
    bool move = false;
#pragma unroll
    for (int half = 0; half < NH; ++half) {
      float m = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) m = fmaxf(m, fmaxf(s[nt][2 * half], s[nt][2 * half + 1]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      top[half] = m;
      move |= m > ref[half] + 8.0f;
    }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int half = 0; half < NH; ++half) {
        const float to = top[half] > ref[half] + 8.0f ? top[half] : ref[half];
        const float g = to == ref[half] ? 1.0f : tc::ex2(ref[half] - to);
        ref[half] = to;
        sum[half] *= g;
        // the output's columns: rows 2c and 2c + 1 of this half, whose factors lanes 8c and 8c + 4 hold
        const float g0 = __shfl_sync(0xffffffffu, g, 8 * c), g1 = __shfl_sync(0xffffffffu, g, 8 * c + 4);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          o[mt][2 * half] *= g0;
          o[mt][2 * half + 1] *= g1;
          od[mt][2 * half] *= g0;
          od[mt][2 * half + 1] *= g1;
        }
      }
    }
    uint32_t pb[NH][4];  // weights of (half, n-tile): keys 8nt + 2c, + 1
#pragma unroll
    for (int half = 0; half < NH; ++half) {
      const float base = (ref[half] == -INFINITY ? 0.0f : ref[half]) - 7.0f;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const float p0 = tc::ex2(s[nt][2 * half] - base), p1 = tc::ex2(s[nt][2 * half + 1] - base);
        sum[half] += p0 + p1;
        pb[half][nt] = tc::cvt_half2(p0, p1);
      }
    }
    const float vsu = vs * code_unit<CODE>();
#pragma unroll
    for (int wd = 0; wd < D / 32; ++wd) {  // four channels of the thread's: output tiles 2wd, 2wd + 1
      float acc[2][NH][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int half = 0; half < NH; ++half)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][half][e] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        // bytes of key pairs interleaved: channel by channel, (key 2c, key 2c + 1)
        const uint32_t x01 = __byte_perm(vr[kk][0][wd], vr[kk][1][wd], 0x5140);
        const uint32_t x23 = __byte_perm(vr[kk][0][wd], vr[kk][1][wd], 0x7362);
        const uint32_t y01 = __byte_perm(vr[kk][2][wd], vr[kk][3][wd], 0x5140);
        const uint32_t y23 = __byte_perm(vr[kk][2][wd], vr[kk][3][wd], 0x7362);
        uint32_t a[2][4];
        codes_f16<CODE>(x01, a[0][0], a[0][1]);
        codes_f16<CODE>(y01, a[0][2], a[0][3]);
        codes_f16<CODE>(x23, a[1][0], a[1][1]);
        codes_f16<CODE>(y23, a[1][2], a[1][3]);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int half = 0; half < NH; ++half)
            mma_16816(acc[m][half], a[m], pb[half][2 * kk], pb[half][2 * kk + 1]);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int half = 0; half < NH; ++half) {
          const int mt = 2 * wd + m;
          o[mt][2 * half] = fmaf(vsu, acc[m][half][0], o[mt][2 * half]);
          o[mt][2 * half + 1] = fmaf(vsu, acc[m][half][1], o[mt][2 * half + 1]);
          od[mt][2 * half] = fmaf(vsu, acc[m][half][2], od[mt][2 * half]);
          od[mt][2 * half + 1] = fmaf(vsu, acc[m][half][3], od[mt][2 * half + 1]);
        }
    }
    if (more) load_v();
  }

  // join the warps
#pragma unroll
  for (int half = 0; half < NH; ++half) {
    sum[half] += __shfl_xor_sync(0xffffffffu, sum[half], 1);
    sum[half] += __shfl_xor_sync(0xffffffffu, sum[half], 2);
    if (c == 0) {
      sm_ref[warp][half * 8 + r] = ref[half];
      sm_sum[warp][half * 8 + r] = sum[half];
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int ch = r * (D / 8) + 2 * mt;
      *reinterpret_cast<float2*>(&sm_o[warp][half * 8 + 2 * c][ch]) = make_float2(o[mt][2 * half], od[mt][2 * half]);
      *reinterpret_cast<float2*>(&sm_o[warp][half * 8 + 2 * c + 1][ch]) =
          make_float2(o[mt][2 * half + 1], od[mt][2 * half + 1]);
    }
  }
  __syncthreads();
  for (int x = tid; x < ROWS * D / 4; x += kFewWarps * 32) {
    const int row = x / (D / 4), ch = (x % (D / 4)) * 4;
    const int i = (row0 + row) / p.G;
    if (i >= sv.q_len) continue;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) m = fmaxf(m, sm_ref[w][row]);
    float l = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float g = sm_ref[w][row] == m ? 1.0f : tc::ex2(sm_ref[w][row] - m);  // (a NaN's sum goes on)
      l += g * sm_sum[w][row];
      const float4 a = *reinterpret_cast<const float4*>(&sm_o[w][row][ch]);
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

// Joins the splits: one warp per row.
template <int D>
__global__ void __launch_bounds__(128) paged_join_kernel(const __grid_constant__ PagedAttnParams p, int rows_pad) {
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int rows = p.n * p.G;
  const int64_t bh = w / rows;
  if (bh >= static_cast<int64_t>(p.B) * p.c.H) return;
  const int row = static_cast<int>(w - bh * rows);
  const int b = static_cast<int>(bh / p.c.H), h = static_cast<int>(bh % p.c.H);
  const SeqView sv = seq_view(p, b);
  if (row / p.G >= sv.q_len) return;
  const int64_t stride = static_cast<int64_t>(p.B) * p.c.H * rows_pad;
  const int64_t at = bh * rows_pad + row;
  float m = -INFINITY;
  for (int s = lane; s < p.splits; s += 32) m = fmaxf(m, p.part_ml[at + s * stride].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.0f;
  const int ch = lane * 4;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s = 0; s < p.splits; ++s) {
    const float2 ml = p.part_ml[at + s * stride];
    const float g = ml.x == m ? 1.0f : tc::ex2(ml.x - m);
    l = fmaf(g, ml.y, l);
    if (ch < D) {
      const float4 a = *reinterpret_cast<const float4*>(p.part_o + (at + s * stride) * D + ch);
      v.x = fmaf(g, a.x, v.x), v.y = fmaf(g, a.y, v.y), v.z = fmaf(g, a.z, v.z), v.w = fmaf(g, a.w, v.w);
    }
  }
  if (ch < D) write_row<D>(p, b, h, row, ch, v, m, l);
}

// Sums of the attention weights: one warp per 32 cached tokens of a (sequence, head), whose
// K codes stay in registers as MMA fragments while the query rows pass by in tiles of 16.
// A token's sum runs over the rows in order, without atomics: results repeat to the bit.
template <int D, int CODE, bool BIAS>
__global__ void __launch_bounds__(kFewWarps * 32) paged_weights_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int KS = D / 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = lane & 3, r = lane >> 2;
  const int groups = (p.c.max_pages + 1) / 2;
  const int bh = blockIdx.x / groups;
  const int b = bh / p.c.H, h = bh - b * p.c.H;
  const int u = (blockIdx.x % groups) * kFewWarps + warp;
  const int slot0 = u * 32;
  const SeqView sv = seq_view(p, b);
  if (slot0 >= sv.len) return;
  const int page = paged_page(p.c, b, u / 2);
  if (page < 0) return;
  const int64_t ph = static_cast<int64_t>(page) * p.c.H + h;
  uint4 kr[4][D / 64];
  load_k<D>(p.c.code[0] + (ph * kPage + (u & 1) * 32) * D, lane, kr);
  const float qk = __ldg(p.c.scale[0] + ph) * p.sigma * code_unit<CODE>() * (BIAS ? 1.0f : kLog2e);
  const float cap_f = BIAS && p.cap > 0.0f ? 2.0f * kLog2e / p.cap : 0.0f;
  const int32_t* pos = p.c.pos ? p.c.pos + ph * kPage + (u & 1) * 32 : nullptr;

  float w[4][2];
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) w[nt][0] = w[nt][1] = 0.0f;
  const int rows = sv.q_len * p.G;
  int row0 = 0;
  // rows before the first that the causal rule lets see this unit (a prefix may let every row see it)
  if (p.causal && !(p.prefix && (p.c.pos || slot0 < sv.prefix)))
    row0 = max(0, slot0 - (sv.len - sv.q_len)) * p.G / 16 * 16;
  for (; row0 < rows; row0 += 16) {
    RowView rv[2];
    bool any = false, whole = true;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      rv[half] = row_view(p, sv, b, h, row0 + half * 8 + r);
      any |= rv[half].hi >= 0 && (pos || rv[half].first < slot0 + 32);
      whole &= rv[half].hi >= slot0 + 32;
    }
    if (!__any_sync(0xffffffffu, any)) continue;
    whole = __all_sync(0xffffffffu, whole);
    uint32_t qa[KS][4];
    float back[2], f[2], base[2];
    load_q<D, 16>(p, sv, b, h, row0, lane, qa, back);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = row0 + half * 8 + r;
      f[half] = qk * back[half];
      base[half] = INFINITY;  // no such row, or one that saw nothing
      if (rv[half].hi >= 0) {
        const float lse = __ldg(p.lse + (static_cast<int64_t>(b) * p.Hq + h * p.G + row % p.G) * p.n + row / p.G);
        if (lse != -INFINITY) base[half] = lse * kLog2e;
      }
    }
    float s[4][4];
    scores_32<D, CODE, 16>(kr, qa, s);
    finish_scores<16, BIAS>(p, sv, rv, f, cap_f, slot0, lane, !whole, pos, s);
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float w0 = base[0] == INFINITY ? 0.0f : tc::ex2(s[nt][e] - base[0]);
        const float w1 = base[1] == INFINITY ? 0.0f : tc::ex2(s[nt][2 + e] - base[1]);
        w[nt][e] += w0 + w1;
      }
  }
#pragma unroll
  for (int nt = 0; nt < 4; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = w[nt][e];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      const int key = nt * 8 + 2 * c + e;
      if (r == 0 && slot0 + key < sv.len) {
        float* at = p.c.weight + ph * kPage + (u & 1) * 32 + key;
        *at = p.accumulate ? *at + x : x;
      }
    }
}

template <typename F>
cudaError_t paged_attn_dispatch(int d, int code, bool bias, F f) {
  using T = std::true_type;
  using N = std::false_type;
  auto by_bias = [&](auto dd, auto cc) { return bias ? f(dd, cc, T{}) : f(dd, cc, N{}); };
  auto by_code = [&](auto dd) {
    return code == kCodeInt8 ? by_bias(dd, std::integral_constant<int, kCodeInt8>{})
                             : by_bias(dd, std::integral_constant<int, kCodeE4m3>{});
  };
  return d == 64 ? by_code(std::integral_constant<int, 64>{}) : by_code(std::integral_constant<int, 128>{});
}

}  // namespace

}  // namespace vq
