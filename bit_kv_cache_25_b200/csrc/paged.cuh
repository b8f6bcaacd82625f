// Paged 8-bit cache: parameters, the code formats, and the two kernels that move
// tokens in and out of it (append: quantize new tokens into pages; read:
// dequantize a range of tokens into dense tensors).
//
// A page holds 64 tokens of every key head; its codes are 8 bits, one float32
// scale per (page, head) and tensor. The value of a code is x^ = code * scale
// (one float32 product).
//   int8: codes -127..127. A page first written with largest magnitude A gets
//         scale max(A / 127, 2^-126).
//   e4m3: scale is a power of two, the smallest with A <= 448 * scale, so
//         dividing by it is exact and the only rounding is the code's own.
// A page that holds tokens already keeps its scale while the new tokens fit
// (A < 127.5 * scale, A <= 448 * scale) and else grows it by the smallest power
// of two that makes them fit, its codes rounded by the same power: the roundings
// of a code's whole life sum to less than one step of its last scale (1/2 + 1/4
// + ...), however often single tokens are appended.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tc_ptx.cuh"
#include "vq_device.cuh"

namespace vq {

constexpr int kPage = 64;              // tokens per page
constexpr uint32_t kDevErrBadPage = 4u;  // a length or page id out of range: the access was skipped

enum PagedCode : int { kCodeInt8 = 0, kCodeE4m3 = 1 };
enum PagedType : int { kTypeBf16 = 0, kTypeF32 = 1, kTypeF16 = 2 };

// The pools and the tables of one call.
struct PagedPool {
  unsigned char* code[2];  // K, V: [num_pages][H][64][D]
  float* scale[2];         // [num_pages][H]
  int32_t* pos;            // [num_pages][H][64] or NULL
  float* weight;           // [num_pages][H][64] or NULL
  const int32_t* table;    // [B][max_pages]
  int H, D;
  int num_pages, max_pages;
};

__device__ __forceinline__ void paged_error() { atomicOr(&g_device_error, kDevErrBadPage); }

// Page id of a sequence's page index; -1 (and the error flag) if either is out of range.
__device__ __forceinline__ int paged_page(const PagedPool& p, int b, int index) {
  if (index < 0 || index >= p.max_pages) {
    paged_error();
    return -1;
  }
  const int id = __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + index);
  if (id < 0 || id >= p.num_pages) {
    paged_error();
    return -1;
  }
  return id;
}

// Cached tokens of sequence b, cut to what its table can hold.
__device__ __forceinline__ int paged_len(const PagedPool& p, const int32_t* lens, int b) {
  const int64_t most = static_cast<int64_t>(p.max_pages) * kPage;
  int len = __ldg(lens + b);
  if (len < 0 || len > most) {
    paged_error();
    len = len < 0 ? 0 : static_cast<int>(most);
  }
  return len;
}

// ---- codes
// Two int8 codes (each xor 0x80; `sel` picks their bytes) as fp16x2: the byte u = code
// + 128 under the high byte 0x64 is the fp16 number 1024 + u, exactly.
__device__ __forceinline__ uint32_t int8_pair_f16(uint32_t flipped, uint32_t sel) {
  const uint32_t v = __byte_perm(flipped, 0x64646464u, sel);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Two e4m3 codes as fp16x2 holding 2^-8 times their values: the code's four exponent
// and three mantissa bits are the low exponent and high mantissa bits of a half
// (exponent biases 7 and 15), subnormals included. The NaN code reads as 480.
__device__ __forceinline__ uint32_t e4m3_pair_f16(uint32_t w, uint32_t sel) {
  const uint32_t v = __byte_perm(w, 0u, sel);  // each code in the high byte of its half
  return (v & 0x80008000u) | ((v & 0x7f007f00u) >> 1);
}
// The four codes of a word as two fp16x2 (codes 0, 1 and 2, 3).
template <int CODE>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (CODE == kCodeInt8) {
    w ^= 0x80808080u;
    lo = int8_pair_f16(w, 0x4140);
    hi = int8_pair_f16(w, 0x4342);
  } else {
    lo = e4m3_pair_f16(w, 0x1404);
    hi = e4m3_pair_f16(w, 0x3424);
  }
}
// The four codes of a word that holds two channels (bytes 0, 1 and 2, 3) of two tokens: channel 0 of both, channel 1.
template <int CODE>
__device__ __forceinline__ void codes_f16_of_two(uint32_t w, uint32_t& even, uint32_t& odd) {
  if (CODE == kCodeInt8) {
    w ^= 0x80808080u;
    even = int8_pair_f16(w, 0x4240);
    odd = int8_pair_f16(w, 0x4341);
  } else {
    even = e4m3_pair_f16(w, 0x2404);
    odd = e4m3_pair_f16(w, 0x3414);
  }
}
// What codes_f16 leaves to the scale.
template <int CODE>
__device__ __forceinline__ constexpr float code_unit() {
  return CODE == kCodeInt8 ? 1.0f : 256.0f;
}

template <int CODE>
__device__ __forceinline__ float code_value(uint32_t byte) {
  if (CODE == kCodeInt8) return static_cast<float>(static_cast<int8_t>(byte));
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(byte & 0xff)));
  return __half2float(__ushort_as_half(static_cast<uint16_t>(h2 & 0xffff)));
}
// The values of two codes (the low half of `pair`).
template <int CODE>
__device__ __forceinline__ void code_values(uint32_t pair, float& lo, float& hi) {
  if (CODE == kCodeInt8) {
    lo = code_value<CODE>(pair & 0xff);
    hi = code_value<CODE>((pair >> 8) & 0xff);
  } else {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(pair)));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    lo = v.x;
    hi = v.y;
  }
}
// {lo, hi} -> two e4m3 codes, nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// ---- 16-byte vectors of the dense tensors
template <int T>
struct PagedVec;
template <>
struct PagedVec<kTypeBf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    const uint32_t w = (&v.x)[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return tc::cvt_bf162(lo, hi); }
  // running maximum of the magnitudes' bits, two values at a time, and that maximum as a float's bits
  static __device__ __forceinline__ void top(const uint4& v, uint32_t& t) {
    t = __vmaxu2(t, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
  }
  static __device__ __forceinline__ uint32_t top_bits(uint32_t t) { return max(t & 0xffffu, t >> 16) << 16; }
};
template <>
struct PagedVec<kTypeF16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    const uint32_t w = (&v.x)[i >> 1];
    return __half2float(__ushort_as_half(static_cast<uint16_t>((i & 1) ? (w >> 16) : (w & 0xffff))));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return tc::cvt_half2(lo, hi); }
  static __device__ __forceinline__ void top(const uint4& v, uint32_t& t) { PagedVec<kTypeBf16>::top(v, t); }
  static __device__ __forceinline__ uint32_t top_bits(uint32_t t) {
    const uint32_t m = max(t & 0xffffu, t >> 16);
    return m > 0x7c00u ? 0x7fffffffu : __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(m))));
  }
};
template <>
struct PagedVec<kTypeF32> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float get(const uint4& v, int i) { return __uint_as_float((&v.x)[i]); }
  static __device__ __forceinline__ void top(const uint4& v, uint32_t& t) {
    t = max(max(t, max(v.x & 0x7fffffffu, v.y & 0x7fffffffu)), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
  }
  static __device__ __forceinline__ uint32_t top_bits(uint32_t t) { return t; }
};

struct PagedAppendParams {
  PagedPool c;
  const void* x[2];
  int64_t sb[2], sh[2], st[2];  // strides in elements
  const int32_t* start;
  const int32_t* counts;        // or NULL: n for every sequence
  const int32_t* pos;           // position of the first new token, or NULL: start
  int B, n, tiles;              // tiles: most pages that n tokens can touch
};

namespace {

constexpr int kAppendThreads = 128;
constexpr float kPagedMost = 8.507059173023462e37f;  // 2^126: larger magnitudes are cut to it

// One CTA per (sequence, head, page touched, tensor). The page's new rows are
// held in registers between the maximum and the encoding, so each input byte is
// read once and each code written once: bound by memory (esize + 1 bytes per
// element; 4 x 4680 tokens of 12 heads in bf16 39 us, 4.4 TB/s). Old codes of the page are only touched when the scale has to grow.
template <int T, int CODE, int D>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  using V = PagedVec<T>;
  constexpr int LPR = D / V::N;                            // lanes per row
  constexpr int RPI = kAppendThreads / LPR;                // rows per CTA load
  constexpr int R = kPage / RPI;
  __shared__ uint32_t red[kAppendThreads / 32];
  const int t = blockIdx.x & 1;
  const int tile = (blockIdx.x >> 1) % p.tiles;
  const int bh = (blockIdx.x >> 1) / p.tiles;
  const int b = bh / p.c.H, h = bh - b * p.c.H;
  const int tid = threadIdx.x;

  const int start = __ldg(p.start + b);
  int cnt = p.counts ? __ldg(p.counts + b) : p.n;
  if (start < 0 || cnt < 0 || cnt > p.n) {
    if (tid == 0) paged_error();
    if (start < 0 || cnt < 0) return;
    cnt = p.n;
  }
  // (start + cnt may pass 2^31: 64-bit)
  const int64_t end = static_cast<int64_t>(start) + cnt;
  const int index = start / kPage + tile;
  const int64_t first = static_cast<int64_t>(index) * kPage;  // token in slot 0
  if (first >= end) return;
  const int lo = first >= start ? 0 : static_cast<int>(start - first);
  const int hi = end - first >= kPage ? kPage : static_cast<int>(end - first);
  const int page = paged_page(p.c, b, index);
  if (page < 0) return;
  const int64_t ph = static_cast<int64_t>(page) * p.c.H + h;

  const typename std::conditional<T == kTypeF32, float, uint16_t>::type* x =
      static_cast<const typename std::conditional<T == kTypeF32, float, uint16_t>::type*>(p.x[t]) +
      b * p.sb[t] + h * p.sh[t];
  const int lane_c = (tid % LPR) * V::N;
  uint4 val[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int slot = i * RPI + tid / LPR;
    val[i] = make_uint4(0, 0, 0, 0);
    if (slot >= lo && slot < hi)
      val[i] = __ldg(reinterpret_cast<const uint4*>(x + (first + slot - start) * p.st[t] + lane_c));
  }
  // largest magnitude as its bits, which order as the magnitudes do; above infinity's: a NaN
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) V::top(val[i], top);
  top = V::top_bits(top);
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) red[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) top = max(top, red[w]);
  float amax = __uint_as_float(top);
  const bool cut = !(amax <= kPagedMost);  // something to cut, or a NaN: once more, value by value
  if (cut) {
    amax = 0.0f;
#pragma unroll 1
    for (int i = 0; i < R; ++i) {
      uint4 v = val[0];
#pragma unroll
      for (int k = 1; k < R; ++k)
        if (k == i) v = val[k];
#pragma unroll
      for (int j = 0; j < V::N; ++j) amax = fmaxf(amax, fabsf(V::get(v, j)));  // a NaN is passed over
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = __float_as_uint(amax);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, __uint_as_float(red[w]));
    amax = fminf(amax, kPagedMost);
  }

  const float old = lo > 0 ? p.c.scale[t][ph] : 0.0f;
  float scale = old;
  int grow = 0;
  if (!(old > 0.0f)) {
    if (CODE == kCodeInt8) {
      scale = amax > 0.0f ? fmaxf(__fdiv_rn(amax, 127.0f), 1.1754943508222875e-38f) : 0.0f;
    } else {
      // smallest e with amax <= 1.75 * 2^(e + 8), from the exponent and mantissa (a subnormal amax gives the floor)
      const uint32_t bits = __float_as_uint(amax);
      const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
      scale = amax > 0.0f ? __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23) : 0.0f;
    }
  } else if (CODE == kCodeInt8) {
    while (__fmaf_rn(127.5f, scale, -amax) <= 0.0f) {  // the sign of the exact difference
      scale *= 2.0f;
      ++grow;
    }
  } else {
    while (__fmul_rn(448.0f, scale) < amax) {
      scale *= 2.0f;
      ++grow;
    }
  }
  __syncthreads();  // every thread has the old scale
  if (tid == 0) p.c.scale[t][ph] = scale;

  unsigned char* code = p.c.code[t] + ph * (kPage * D);
  if (grow > 0) {  // the page's older codes, by the same power of two
    const float f = grow > 126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(127 - grow) << 23);
    for (int i = tid; i < lo * (D / 4); i += kAppendThreads) {
      uint32_t* w = reinterpret_cast<uint32_t*>(code) + i;
      const uint32_t o = *w;
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = code_value<CODE>((o >> (8 * j)) & 0xff) * f;
      uint32_t r = 0;
      if (CODE == kCodeInt8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r |= (static_cast<uint32_t>(__float2int_rn(v[j])) & 0xff) << (8 * j);
      } else {
        r = e4m3_pair(v[0], v[1]) | (e4m3_pair(v[2], v[3]) << 16);
      }
      *w = r;
    }
  }

  // scale >= 2^-126, so its reciprocal is finite; a scale of 0 writes codes of 0 (+0)
  const float inv = scale > 0.0f ? __fdiv_rn(1.0f, scale) : 0.0f;
  const float half = 0.5f * scale;
  const bool rare = cut || !(scale > 0.0f);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int slot = i * RPI + tid / LPR;
    if (slot < lo || slot >= hi) continue;
    uint32_t out[V::N / 4];
#pragma unroll
    for (int g = 0; g < V::N / 4; ++g) {
      float xv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        xv[j] = V::get(val[i], 4 * g + j);
        if (rare) xv[j] = scale > 0.0f && xv[j] == xv[j] ? fminf(fmaxf(xv[j], -kPagedMost), kPagedMost) : 0.0f;
      }
      if (CODE == kCodeInt8) {
        // x * inv rounded by 1.5 * 2^23, then checked: x - k * scale is exact here, so a
        // product that fell on the wrong side of a half (or a tie) shows in it
        float k[4], tt[4];
        bool off = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          tt[j] = __fmaf_rn(xv[j], inv, 12582912.0f);
          k[j] = tt[j] - 12582912.0f;
          off |= fabsf(__fmaf_rn(-k[j], scale, xv[j])) >= half;  // (remainders are multiples of 2^-149: none lies between half and its float)
        }
        if (off) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float rem = __fmaf_rn(-k[j], scale, xv[j]);
            const bool odd = (__float_as_uint(tt[j]) & 1u) != 0;
            // (twice the remainder: half of a scale below 2^-125 may be no float)
            if (fabsf(rem + rem) > scale || (fabsf(rem + rem) == scale && odd)) tt[j] += rem > 0.0f ? 1.0f : -1.0f;
          }
        }
        uint32_t a = __byte_perm(__float_as_uint(tt[0]), __float_as_uint(tt[1]), 0x0040);
        uint32_t c = __byte_perm(__float_as_uint(tt[2]), __float_as_uint(tt[3]), 0x0040);
        out[g] = __byte_perm(a, c, 0x5410);
      } else {
        out[g] = e4m3_pair(xv[0] * inv, xv[1] * inv) | (e4m3_pair(xv[2] * inv, xv[3] * inv) << 16);
      }
    }
    unsigned char* dst = code + slot * D + lane_c;
    if (V::N == 8)
      *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[V::N / 4 - 1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = out[0];
  }
  if (t == 0 && tid >= lo && tid < hi) {
    if (p.c.pos) p.c.pos[ph * kPage + tid] = (p.pos ? __ldg(p.pos + b) : start) + static_cast<int>(first + tid - start);
    if (p.c.weight) p.c.weight[ph * kPage + tid] = 0.0f;
  }
}

}  // namespace

struct PagedReadParams {
  PagedPool c;
  void* out[2];
  int64_t sb[2], sh[2], st[2];
  const int32_t* start;
  const int32_t* counts;
  int B, n, tiles;
};

namespace {

// One CTA per (sequence, head, 64 tokens, tensor): they lie in one page or two. All loads
// of a thread (eight codes a row) are issued before the first is used; one 16-byte store a
// row (two for float32). Bound by memory (8 x 9360 tokens of 12 heads to bf16 122 us, 5.6 TB/s).
template <int T, int CODE, int D>
__global__ void __launch_bounds__(128) paged_read_kernel(const __grid_constant__ PagedReadParams p) {
  constexpr int LPR = D / 8, RPI = 128 / LPR, R = kPage / RPI;
  const int t = blockIdx.x & 1;
  const int tile = (blockIdx.x >> 1) % p.tiles;
  const int bh = (blockIdx.x >> 1) / p.tiles;
  const int b = bh / p.c.H, h = bh - b * p.c.H;
  const int start = __ldg(p.start + b);
  int cnt = p.counts ? __ldg(p.counts + b) : p.n;
  if (start < 0 || cnt < 0 || cnt > p.n) {
    if (threadIdx.x == 0) paged_error();
    if (start < 0 || cnt < 0) return;
    cnt = p.n;
  }
  const int rows = min(cnt - tile * kPage, kPage);
  if (rows <= 0) return;
  const int64_t first = static_cast<int64_t>(start) + tile * kPage;
  const int off = static_cast<int>(first % kPage);
  const int64_t index = first / kPage;
  // rows below `turn` are in the first page, the others in the next; (a page index past the table is an error)
  const int turn = kPage - off;
  int64_t ph[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ph[i] = -1;
    if (i == 0 || rows > turn) {
      const int page = paged_page(p.c, b, index + i < p.c.max_pages ? static_cast<int>(index + i) : -1);
      if (page >= 0) ph[i] = static_cast<int64_t>(page) * p.c.H + h;
    }
  }
  const float s0 = ph[0] >= 0 ? __ldg(p.c.scale[t] + ph[0]) : 0.0f, s1 = ph[1] >= 0 ? __ldg(p.c.scale[t] + ph[1]) : 0.0f;
  const int c = (threadIdx.x % LPR) * 8, r0 = threadIdx.x / LPR;
  uint2 w[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = i * RPI + r0;
    const int64_t page = row < turn ? ph[0] : ph[1];
    w[i] = make_uint2(0, 0);
    if (row < rows && page >= 0)
      w[i] = __ldg(reinterpret_cast<const uint2*>(p.c.code[t] + (page * kPage + ((off + row) & (kPage - 1))) * D + c));
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = i * RPI + r0;
    if (row >= rows || (row < turn ? ph[0] : ph[1]) < 0) continue;
    const float s = row < turn ? s0 : s1;
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      code_values<CODE>(((j < 2 ? w[i].x : w[i].y) >> (16 * (j & 1))) & 0xffffu, v[2 * j], v[2 * j + 1]);
      v[2 * j] = __fmul_rn(v[2 * j], s);
      v[2 * j + 1] = __fmul_rn(v[2 * j + 1], s);
    }
    const int64_t at = b * p.sb[t] + h * p.sh[t] + static_cast<int64_t>(tile * kPage + row) * p.st[t] + c;
    if constexpr (T == kTypeF32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out[t]) + at);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      using V = PagedVec<T>;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out[t]) + at) =
          make_uint4(V::pack(v[0], v[1]), V::pack(v[2], v[3]), V::pack(v[4], v[5]), V::pack(v[6], v[7]));
    }
  }
}

template <typename F>
cudaError_t paged_dispatch(int type, int code, int d, F f) {
  // f(type tag, code tag, head_dim tag) for the combinations that exist
  auto by_d = [&](auto t, auto c) {
    return d == 64 ? f(t, c, std::integral_constant<int, 64>{}) : f(t, c, std::integral_constant<int, 128>{});
  };
  auto by_c = [&](auto t) {
    return code == kCodeInt8 ? by_d(t, std::integral_constant<int, kCodeInt8>{})
                             : by_d(t, std::integral_constant<int, kCodeE4m3>{});
  };
  if (type == kTypeBf16) return by_c(std::integral_constant<int, kTypeBf16>{});
  if (type == kTypeF16) return by_c(std::integral_constant<int, kTypeF16>{});
  return by_c(std::integral_constant<int, kTypeF32>{});
}

}  // namespace

inline cudaError_t launch_paged_append(const PagedAppendParams& p, int type, int code, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.c.H * p.tiles * 2);
  return paged_dispatch(type, code, p.c.D, [&](auto t, auto c, auto d) {
    paged_append_kernel<t(), c(), d()><<<grid, kAppendThreads, 0, stream>>>(p);
    return cudaGetLastError();
  });
}

inline cudaError_t launch_paged_read(const PagedReadParams& p, int type, int code, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.c.H * p.tiles * 2);
  return paged_dispatch(type, code, p.c.D, [&](auto t, auto c, auto d) {
    paged_read_kernel<t(), c(), d()><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
  });
}

}  // namespace vq
