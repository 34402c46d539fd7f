// gc_act8.cuh -- the 8-bit checkpoint format of an activation, and typed loads
// and stores of eight consecutive columns, shared by the kernels of the
// backward pass (gc_ckpt.cu, gc_norm.cu, gc_wgrad.cu).
//
// Format (include/gc.h): groups of 32 consecutive columns of a row share one
// scale byte B = biased binary32 exponent of the largest magnitude, plus one;
// an element is sign << 7 | m, m = min(127, rint(|x| * 2^(134 - B))), and
// stands for +-m * 2^(B - 134).  The step is a power of two, so
// |x| * 2^(134 - B) is exact (the code is decided by one rounding, the same
// on every machine) and a restored value, 7 bits times a power of two, is
// exact in binary32, in bf16 and, for values that came from fp16, in fp16.
//
// Work unit: a chunk of 8 consecutive columns per thread, so that the four
// threads of a group of 32 are neighbours in a warp.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gc_internal.cuh"

namespace gc {

constexpr int kChunk = 8;     // columns of one thread's unit
constexpr int kActGroup = 32; // columns that share a scale byte

inline int64_t ckpt_codes_pitch(int64_t cols) { return round_up(cols, kActGroup); }
inline int64_t ckpt_scales_pitch(int64_t cols) {
  return round_up(ceil_div(cols, (int64_t)kActGroup), 16);
}

// ---------------------------------------------------------------------------
// Typed chunks.  A chunk stays in its own type (Raw) until it is used: 4
// registers for the 16-bit types.
// ---------------------------------------------------------------------------
template <int DT>
struct Elem;

template <>
struct Elem<GC_F32> {
  using T = float;
  struct Raw { uint4 a, b; };
  static __device__ __forceinline__ void zero(Raw& r) {
    r.a = make_uint4(0, 0, 0, 0);
    r.b = make_uint4(0, 0, 0, 0);
  }
  static __device__ __forceinline__ void load(Raw& r, const T* p) {
    r.a = __ldg(reinterpret_cast<const uint4*>(p));
    r.b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  static __device__ __forceinline__ void store(T* p, const Raw& r) {
    reinterpret_cast<uint4*>(p)[0] = r.a;
    reinterpret_cast<uint4*>(p)[1] = r.b;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float v[8]) {
    v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y);
    v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
    v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y);
    v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
  }
  static __device__ __forceinline__ void pack(Raw& r, const float v[8]) {
    r.a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3]));
    r.b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                     __float_as_uint(v[7]));
  }
  static __device__ __forceinline__ float to_float(T x) { return x; }
  static __device__ __forceinline__ T from_float(float x) { return x; }
};

template <>
struct Elem<GC_BF16> {
  using T = __nv_bfloat16;
  using Raw = uint4;
  static __device__ __forceinline__ void zero(Raw& r) { r = make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ void load(Raw& r, const T* p) {
    r = __ldg(reinterpret_cast<const uint4*>(p));
  }
  static __device__ __forceinline__ void store(T* p, const Raw& r) {
    *reinterpret_cast<uint4*>(p) = r;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float v[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void pack(Raw& r, const float v[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float to_float(T x) { return __bfloat162float(x); }
  static __device__ __forceinline__ T from_float(float x) { return __float2bfloat16_rn(x); }
};

template <>
struct Elem<GC_F16> {
  using T = __half;
  using Raw = uint4;
  static __device__ __forceinline__ void zero(Raw& r) { r = make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ void load(Raw& r, const T* p) {
    r = __ldg(reinterpret_cast<const uint4*>(p));
  }
  static __device__ __forceinline__ void store(T* p, const Raw& r) {
    *reinterpret_cast<uint4*>(p) = r;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float v[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void pack(Raw& r, const float v[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float to_float(T x) { return __half2float(x); }
  static __device__ __forceinline__ T from_float(float x) { return __float2half_rn(x); }
};

// Eight columns starting at p of which the first `valid` (1..8) exist; the
// rest read as zero.  VEC: p is 16-byte aligned.
template <int DT, bool VEC>
__device__ __forceinline__ void load_chunk(float v[8], const typename Elem<DT>::T* p, int valid) {
  using E = Elem<DT>;
  if (VEC && valid >= kChunk) {
    typename E::Raw r;
    E::load(r, p);
    E::unpack(r, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < kChunk; ++i) v[i] = i < valid ? E::to_float(p[i]) : 0.0f;
}

template <int DT, bool VEC>
__device__ __forceinline__ void store_chunk(typename Elem<DT>::T* p, const float v[8], int valid) {
  using E = Elem<DT>;
  if (VEC && valid >= kChunk) {
    typename E::Raw r;
    E::pack(r, v);
    E::store(p, r);
    return;
  }
#pragma unroll
  for (int i = 0; i < kChunk; ++i)
    if (i < valid) p[i] = E::from_float(v[i]);
}

// ---------------------------------------------------------------------------
// The format.
// ---------------------------------------------------------------------------

// Largest magnitude (as bits; a NaN compares above infinity) of a thread's
// chunk, then of the group's four threads.  All 32 lanes take part.
__device__ __forceinline__ uint32_t group_max_bits(const float v[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kChunk; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return m;
}

__device__ __forceinline__ uint32_t scale_byte(uint32_t max_bits) {
  const uint32_t e = max_bits >> 23;
  return e < 7u ? 0u : (e >= 254u ? 255u : e + 1u);
}

// Codes of four values at scale byte b.  |x| * up < 128 + 2^23 addition: the
// sum's low mantissa bits are the product rounded half to even.
__device__ __forceinline__ uint32_t encode4(const float v[4], float up) {
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = __float_as_uint(__fadd_rn(fminf(__fmul_rn(fabsf(v[i]), up), 127.0f), 8388608.0f));
  const uint32_t lo = __byte_perm(q[0], q[1], 0x0040), hi = __byte_perm(q[2], q[3], 0x0040);
  const uint32_t m = __byte_perm(lo, hi, 0x5410);
  const uint32_t slo = __byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x0073);
  const uint32_t shi = __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x0073);
  const uint32_t sign = __byte_perm(slo, shi, 0x5410);
  const uint32_t nonzero = m + 0x7F7F7F7Fu;  // bit 7 of each byte: m != 0
  return m | (sign & nonzero & 0x80808080u);
}

__device__ __forceinline__ uint2 encode8(const float v[8], uint32_t b) {
  if (b == 0u || b == 255u) return make_uint2(0u, 0u);
  const float up = __uint_as_float((261u - b) << 23);  // 2^(134 - b)
  return make_uint2(encode4(v, up), encode4(v + 4, up));
}

// The value of the code in byte i of w: the binary32 word with sign, exponent
// b and the seven bits m on top of its mantissa is +-(128 + m) * 2^(b - 134);
// taking +-128 * 2^(b - 134) off it is exact.  b == 255 gives inf - inf = NaN.
__device__ __forceinline__ float decode1(uint32_t w, int i, uint32_t bexp) {
  const uint32_t c = __byte_perm(w, 0u, 0x0044u | ((uint32_t)i << 8) | ((uint32_t)i << 12));
  // c = byte i in bytes 3 and 2 (byte 0, 1 from the zero word)
  const uint32_t s = c & 0x80000000u;
  const uint32_t x = s | bexp | (c & 0x007F0000u);
  return __fsub_rn(__uint_as_float(x), __uint_as_float(s | bexp));
}

__device__ __forceinline__ void decode8(float v[8], uint2 w, uint32_t b) {
  const uint32_t bexp = b << 23;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = decode1(w.x, i, bexp);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[4 + i] = decode1(w.y, i, bexp);
}

}  // namespace gc
