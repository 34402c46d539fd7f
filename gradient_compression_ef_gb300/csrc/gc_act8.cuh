// gc_act8.cuh -- the 8-bit checkpoint format of an activation, and typed loads
// and stores of 16 consecutive bytes of a row, shared by the kernels of the
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
// Work unit: 16 bytes of a row (8 columns of a 16-bit type, 4 of fp32) per
// thread, so that every load and store of a warp is one run of 512 bytes and
// the threads of a group of 32 columns (4 or 8) are neighbours in a warp.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gc_internal.cuh"

namespace gc {

constexpr int kActGroup = 32;  // columns that share a scale byte

inline int64_t ckpt_codes_pitch(int64_t cols) { return round_up(cols, kActGroup); }
inline int64_t ckpt_scales_pitch(int64_t cols) {
  return round_up(ceil_div(cols, (int64_t)kActGroup), 16);
}

// ---------------------------------------------------------------------------
// Typed units: 16 bytes as they lie in memory, unpacked to V fp32 values.
// ---------------------------------------------------------------------------
template <int DT>
struct Elem;

template <>
struct Elem<GC_F32> {
  using T = float;
  static constexpr int V = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[V]) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[V]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};

template <>
struct Elem<GC_BF16> {
  using T = __nv_bfloat16;
  static constexpr int V = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[V]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[V]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Elem<GC_F16> {
  using T = __half;
  static constexpr int V = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[V]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[V]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// A unit as pairs, for the packed fp32 instructions.
template <int DT>
__device__ __forceinline__ void unpack2(const uint4& r, float2 (&v)[Elem<DT>::V / 2]) {
  float f[Elem<DT>::V];
  Elem<DT>::unpack(r, f);
#pragma unroll
  for (int i = 0; i < Elem<DT>::V / 2; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
}
template <int DT>
__device__ __forceinline__ uint4 pack2(const float2 (&v)[Elem<DT>::V / 2]) {
  float f[Elem<DT>::V];
#pragma unroll
  for (int i = 0; i < Elem<DT>::V / 2; ++i) {
    f[2 * i] = v[i].x;
    f[2 * i + 1] = v[i].y;
  }
  return Elem<DT>::pack(f);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

constexpr int elem_size(int dtype) { return dtype == GC_F32 ? 4 : 2; }
inline bool row_aligned(int64_t ld, int dtype) { return ld * elem_size(dtype) % 16 == 0; }

// ---------------------------------------------------------------------------
// Runs of units.  A warp's run is U times 32 consecutive units of a row, from
// byte `at` (a multiple of 512) of the row on; lane l has units l, l + 32, ...
// Columns past the row's `bytes` read as zero and are not stored.  Inside the
// row (`inner`, the same in the whole warp: at + 512 U <= bytes, 16 less where
// rows are not aligned) nothing is checked and every address is one base plus
// a constant.
//
// Rows that start anywhere are read and written in the aligned 16-byte pieces
// that cover the run; lanes exchange neighbouring pieces and cut their units
// from them.  A piece may hold bytes of the row before (never from before the
// matrix: its first row is aligned) or of the row after; nothing is read past
// `end`, the matrix's end, and pieces that the run does not fill are stored
// by elements.
// ---------------------------------------------------------------------------

// Elements [0, n) of 16 bytes, one by one.
template <int DT>
__device__ __forceinline__ uint4 load_some(const char* p, int n) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (DT == GC_F32) {
      if (i < n) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
      if (2 * i < n) w[i] = h[2 * i];
      if (2 * i + 1 < n) w[i] |= (uint32_t)h[2 * i + 1] << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements [lo, hi) of 16 bytes, one by one.
template <int DT>
__device__ __forceinline__ void store_some(char* p, const uint4& r, int lo, int hi) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (DT == GC_F32) {
      if (i >= lo && i < hi) reinterpret_cast<uint32_t*>(p)[i] = w[i];
    } else {
      uint16_t* h = reinterpret_cast<uint16_t*>(p);
      if (2 * i >= lo && 2 * i < hi) h[2 * i] = (uint16_t)w[i];
      if (2 * i + 1 >= lo && 2 * i + 1 < hi) h[2 * i + 1] = (uint16_t)(w[i] >> 16);
    }
  }
}

// 16 of the 32 bytes lo ++ hi, from byte `shift` (0..15, even; the same in
// the whole warp) on.
__device__ __forceinline__ uint4 funnel(const uint4& lo, const uint4& hi, uint32_t shift) {
  uint32_t w[5];
  switch (shift >> 2) {
    case 0: w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w; w[4] = hi.x; break;
    case 1: w[0] = lo.y; w[1] = lo.z; w[2] = lo.w; w[3] = hi.x; w[4] = hi.y; break;
    case 2: w[0] = lo.z; w[1] = lo.w; w[2] = hi.x; w[3] = hi.y; w[4] = hi.z; break;
    default: w[0] = lo.w; w[1] = hi.x; w[2] = hi.y; w[3] = hi.z; w[4] = hi.w; break;
  }
  const uint32_t sh = (shift & 3u) * 8u;
  return make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh),
                    __funnelshift_r(w[2], w[3], sh), __funnelshift_r(w[3], w[4], sh));
}

__device__ __forceinline__ uint4 shfl4(const uint4& v, int from) {
  return make_uint4(__shfl_sync(0xffffffffu, v.x, from), __shfl_sync(0xffffffffu, v.y, from),
                    __shfl_sync(0xffffffffu, v.z, from), __shfl_sync(0xffffffffu, v.w, from));
}

// The unit with the columns from byte `left` on set to zero.
__device__ __forceinline__ void cut_unit(uint4& r, int64_t left) {
  if (left >= 16) return;
  uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (left <= 4 * i) w[i] = 0u;
    else if (left == 4 * i + 2) w[i] &= 0xFFFFu;
  }
  r = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DT, bool ALIGNED, int U>
__device__ __forceinline__ void load_run(uint4 (&r)[U], const char* row, uint32_t at, bool inner,
                                         int64_t bytes, const char* end) {
  constexpr int E = elem_size(DT);
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t mis = ALIGNED ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
  const int64_t o = (int64_t)at + lane * 16u - mis;  // the first piece's place in the row
  const char* p = row + o;
  if (inner) {
#pragma unroll
    for (int i = 0; i < U; ++i) r[i] = __ldg(reinterpret_cast<const uint4*>(p + i * 512));
  } else if (ALIGNED && (bytes & 15) == 0) {  // whole units
#pragma unroll
    for (int i = 0; i < U; ++i)
      r[i] = o + i * 512 < bytes ? __ldg(reinterpret_cast<const uint4*>(p + i * 512))
                                 : make_uint4(0u, 0u, 0u, 0u);
    return;
  } else {
    const int64_t e = end - row;
    int cut = -1;  // the piece that the matrix ends in
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t oi = o + i * 512;
      r[i] = make_uint4(0u, 0u, 0u, 0u);
      if (oi < bytes) {
        if (oi + 16 <= e) r[i] = __ldg(reinterpret_cast<const uint4*>(p + i * 512));
        else cut = i;
      }
    }
    if (cut >= 0) {
      const uint4 v = load_some<DT>(p + cut * 512, (int)(e - o - cut * 512) / E);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (i == cut) r[i] = v;
    }
  }
  if (!ALIGNED && mis) {
    uint4 last = make_uint4(0u, 0u, 0u, 0u);  // the piece behind the run, for lane 31
    const int64_t ol = o + (U - 1) * 512 + 16;
    if (lane == 31u && (inner || ol < bytes)) {
      if (inner || ol + 16 <= end - row) last = __ldg(reinterpret_cast<const uint4*>(row + ol));
      else last = load_some<DT>(row + ol, (int)(end - row - ol) / E);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      // the next lane's piece; lane 31's next is lane 0's of the next segment
      const uint4 v = (i + 1 < U && lane == 0u) ? r[i + 1 < U ? i + 1 : i] : r[i];
      uint4 n = shfl4(v, (int)((lane + 1u) & 31u));
      if (i == U - 1 && lane == 31u) n = last;
      r[i] = funnel(r[i], n, mis);
    }
  }
  if (!inner) {
#pragma unroll
    for (int i = 0; i < U; ++i) cut_unit(r[i], bytes - at - i * 512 - lane * 16);
  }
}

template <int DT, bool ALIGNED, int U>
__device__ __forceinline__ void store_run(char* row, uint32_t at, bool inner, int64_t bytes,
                                          const uint4 (&r)[U]) {
  constexpr int E = elem_size(DT);
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t mis = ALIGNED ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
  const int64_t o = (int64_t)at + lane * 16u - mis;
  char* p = row + o;
  if (ALIGNED || mis == 0u) {
    if (inner) {
#pragma unroll
      for (int i = 0; i < U; ++i) *reinterpret_cast<uint4*>(p + i * 512) = r[i];
      return;
    }
    if ((bytes & 15) == 0) {  // whole units
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (o + i * 512 < bytes) *reinterpret_cast<uint4*>(p + i * 512) = r[i];
      return;
    }
    int cut = -1;  // the unit that the row ends in
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t left = bytes - o - i * 512;
      if (left >= 16) {
        *reinterpret_cast<uint4*>(p + i * 512) = r[i];
      } else if (left > 0) {
        cut = i;
        v = r[i];
      }
    }
    if (cut >= 0) store_some<DT>(p + cut * 512, v, 0, (int)(bytes - o - cut * 512) / E);
    return;
  }
  int cut = -1;  // the piece that the row ends in
  uint4 v = make_uint4(0u, 0u, 0u, 0u), first = v;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    // the lane before's unit; lane 0's is lane 31's of the segment before
    const uint4 u = (i > 0 && lane == 31u) ? r[i > 0 ? i - 1 : 0] : r[i];
    const uint4 piece = funnel(shfl4(u, (int)((lane + 31u) & 31u)), r[i], 16u - mis);
    const int64_t left = bytes - o - i * 512;
    if (i == 0 && lane == 0u) {
      first = piece;
    } else if (inner || left >= 16) {
      *reinterpret_cast<uint4*>(p + i * 512) = piece;
    } else if (left > 0) {
      cut = i;
      v = piece;
    }
  }
  if (cut >= 0) store_some<DT>(p + cut * 512, v, 0, (int)(bytes - o - cut * 512) / E);
  // The two pieces that the run shares with its neighbours, an element per
  // lane: lane 0's first piece by the lanes of the lower half, the piece
  // behind lane 31's last unit, which holds that unit's end, by the upper's.
  const uint4 tail = funnel(r[U - 1], r[U - 1], 16u - mis);
  const uint4 q = shfl4(lane == 0u ? first : tail, lane < 16u ? 0 : 31);
  const uint32_t k = lane & 15u, w = k * E / 4;  // the lane's element, its word
  if (k * E < 16u) {
    const uint32_t word = w == 0u ? q.x : w == 1u ? q.y : w == 2u ? q.z : q.w;
    const bool upper = lane >= 16u;
    // its place in the row
    const int64_t c = (int64_t)at - mis + (upper ? U * 512 : 0) + k * E;
    if (upper == ((int)(k * E) < (int)mis) && c < bytes) {
      if (DT == GC_F32) *reinterpret_cast<uint32_t*>(row + c) = word;
      else *reinterpret_cast<uint16_t*>(row + c) = (uint16_t)(k & 1u ? word >> 16 : word);
    }
  }
}

// One unit per lane, `off` being the lane's byte in the row (a whole warp's
// units are consecutive).
template <int DT, bool ALIGNED>
__device__ __forceinline__ uint4 load_unit(const char* row, int64_t off, int64_t bytes,
                                           const char* end) {
  uint4 r[1];
  load_run<DT, ALIGNED>(r, row, (uint32_t)off - (threadIdx.x & 31u) * 16u, false, bytes, end);
  return r[0];
}
template <int DT, bool ALIGNED>
__device__ __forceinline__ void store_unit(char* row, int64_t off, int64_t bytes,
                                           const uint4& r) {
  const uint4 u[1] = {r};
  store_run<DT, ALIGNED>(row, (uint32_t)off - (threadIdx.x & 31u) * 16u, false, bytes, u);
}

// ---------------------------------------------------------------------------
// The format.
// ---------------------------------------------------------------------------

// Largest magnitude of a unit's group, as binary32 bits (a NaN compares above
// infinity).  16-bit types compare their magnitude bits two at a time.  All
// 32 lanes take part.
template <int DT>
__device__ __forceinline__ uint32_t group_max_bits(const uint4& r) {
  if (DT == GC_F32) {
    uint32_t m = max(max(r.x & 0x7FFFFFFFu, r.y & 0x7FFFFFFFu),
                     max(r.z & 0x7FFFFFFFu, r.w & 0x7FFFFFFFu));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  }
  uint32_t m = __vmaxu2(__vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu),
                        __vmaxu2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  const uint32_t h = max(m & 0xFFFFu, m >> 16);
  if (DT == GC_BF16) return h << 16;
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
}

__device__ __forceinline__ uint32_t scale_byte(uint32_t max_bits) {
  const uint32_t e = max_bits >> 23;
  return e < 7u ? 0u : (e >= 254u ? 255u : e + 1u);
}

// Codes of four values, up = 2^(134 - B), from the values and the bytes that
// hold their signs.  The fused multiply-add rounds |x| * up + 2^23 once, to
// the product rounded half to even in its low byte; 128 (from above 127.5)
// becomes 127.
__device__ __forceinline__ uint32_t encode4(const float* v, uint32_t signs, float up) {
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const float2 m = __ffma2_rn(make_float2(fabsf(v[i]), fabsf(v[i + 1])), both(up),
                                both(8388608.0f));
    q[i] = __float_as_uint(m.x);
    q[i + 1] = __float_as_uint(m.y);
  }
  uint32_t m = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040),
                           0x5410);
  m -= (m >> 7) & 0x01010101u;
  const uint32_t nonzero = m + 0x7F7F7F7Fu;  // bit 7 of each byte: m != 0
  return m | (signs & nonzero & 0x80808080u);
}

// A unit's codes (one word for fp32, two for 16-bit types) from its bytes
// and its values.
template <int DT>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint4& r,
                                            const float (&v)[Elem<DT>::V], uint32_t b) {
  const bool empty = b == 0u || b == 255u;
  const float up = __uint_as_float((261u - b) << 23);
  if (DT == GC_F32) {
    const uint32_t s = __byte_perm(__byte_perm(r.x, r.y, 0x0073), __byte_perm(r.z, r.w, 0x0073),
                                   0x5410);
    *reinterpret_cast<uint32_t*>(p) = empty ? 0u : encode4(v, s, up);
  } else {
    const uint32_t c0 = encode4(v, __byte_perm(r.x, r.y, 0x7531), up);
    const uint32_t c1 = encode4(v + Elem<DT>::V - 4, __byte_perm(r.z, r.w, 0x7531), up);
    *reinterpret_cast<uint2*>(p) = empty ? make_uint2(0u, 0u) : make_uint2(c0, c1);
  }
}

template <int V>
struct Codes {
  uint32_t w[V / 4];
};
template <int V>
__device__ __forceinline__ Codes<V> load_codes(const uint8_t* p) {
  Codes<V> c;
  if (V == 4) c.w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  else {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    c.w[0] = u.x;
    c.w[V / 4 - 1] = u.y;
  }
  return c;
}

// Two codes (the bytes that `sel` puts twice each into the halves) as bf16:
// sign, exponent B and the seven bits m make +-(128 + m) 2^(B - 134); taking
// +-128 2^(B - 134) off is exact.  bexp: B in both exponents; B = 255 gives
// inf - inf = NaN.
__device__ __forceinline__ uint32_t decode2(uint32_t w, uint32_t sel, uint32_t bexp) {
  const uint32_t v = __byte_perm(w, 0u, sel);
  const uint32_t x = (v & 0x807F807Fu) | bexp, c = (v & 0x80008000u) | bexp;
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(c));
  return d;
}

template <int V>
__device__ __forceinline__ void decode(float2 (&v)[V / 2], const Codes<V>& c, uint32_t b) {
  const uint32_t bexp = b * 0x00800080u;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const uint32_t d = decode2(c.w[i / 2], i & 1 ? 0x3322u : 0x1100u, bexp);
    v[i] = make_float2(__uint_as_float(d << 16), __uint_as_float(d & 0xFFFF0000u));
  }
}
template <int V>
__device__ __forceinline__ void decode(float (&v)[V], const Codes<V>& c, uint32_t b) {
  float2 p[V / 2];
  decode<V>(p, c, b);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    v[2 * i] = p[i].x;
    v[2 * i + 1] = p[i].y;
  }
}

}  // namespace gc
