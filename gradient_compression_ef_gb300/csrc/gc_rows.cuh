// gc_rows.cuh -- what the kernels that walk over rows share (gc_norm.cu,
// gc_rms.cu): parameters per column, sums over the threads of a row, rows in
// a ring of stages in shared memory.
#pragma once

#include "gc_act8.cuh"
#include "gc_sm100.cuh"

namespace gc {

// V parameters from column c on; `fill` where there is no vector or column.
template <int V>
__device__ __forceinline__ void load_params(float (&v)[V], const void* p, int ptype, int64_t c,
                                            int64_t cols, float fill) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = fill;
  if (!p) return;
  if (ptype == GC_F32) {
    const float* q = static_cast<const float*>(p) + c;
    if (c + V <= cols) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(q + i));
        v[i] = f.x;
        v[i + 1] = f.y;
        v[i + 2] = f.z;
        v[i + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < cols) v[i] = q[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i < cols)
        v[i] = ptype == GC_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c + i])
                                : __half2float(static_cast<const __half*>(p)[c + i]);
  }
}

// Sums over the threads of a row: the warp's, or the block's (one barrier;
// `turn` alternates the two slots, so the next sum needs no barrier before
// it writes).
template <bool WARP>
struct RowSum {
  float2 (*slot)[32];
  int turn = 0;
  __device__ __forceinline__ float2 operator()(float a, float b) {
    a = warp_allsum(a);
    b = warp_allsum(b);
    if (WARP) return make_float2(a, b);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0) slot[turn][warp] = make_float2(a, b);
    __syncthreads();
    const float2 v = lane < nw ? slot[turn][lane] : make_float2(0.0f, 0.0f);
    turn ^= 1;
    return make_float2(warp_allsum(v.x), warp_allsum(v.y));
  }
  __device__ __forceinline__ float operator()(float a) {
    a = warp_allsum(a);
    if (WARP) return a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0) slot[turn][warp].x = a;
    __syncthreads();
    const float v = lane < nw ? slot[turn][lane].x : 0.0f;
    turn ^= 1;
    return warp_allsum(v);
  }
};

// Keeps a unit packed between the passes over a row: without it the compiler
// unpacks once and holds every value in fp32, at twice the registers.
__device__ __forceinline__ void keep_packed(uint4& r) {
  asm volatile("" : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)::"memory");
}

// A thread's V parameters of unit i, in shared memory.
template <int V>
__device__ __forceinline__ void lds_params(float2 (&g)[V / 2], uint32_t at) {
#pragma unroll
  for (int j = 0; j < V; j += 4) {
    const float4 f = sm100::lds128(at + j * 4);
    g[j / 2] = make_float2(f.x, f.y);
    g[j / 2 + 1] = make_float2(f.z, f.w);
  }
}

// ---------------------------------------------------------------------------
// Rows through a ring of stages in shared memory, which bulk copies fill.
// ---------------------------------------------------------------------------
constexpr long long kWaitCycles = 4000000000ll;  // bound on each wait: ~2 s

// Copies a row's aligned 16-byte pieces to dst and returns the bytes that the
// stage's barrier will see.  The last piece of the matrix's last row may
// reach past the matrix: what is left of it is copied here, by elements.
template <int DT>
__device__ __forceinline__ uint32_t bulk_size(const char* row, int64_t bytes, const char* end,
                                              char* dst) {
  const char* p = row - (reinterpret_cast<uintptr_t>(row) & 15u);
  int64_t n = (row + bytes - p + 15) & ~15ll;
  if (p + n > end) {
    const int64_t whole = (end - p) & ~15ll;
    using T = typename Elem<DT>::T;
    for (int64_t i = whole; i < end - p; i += elem_size(DT))
      *reinterpret_cast<T*>(dst + i) = *reinterpret_cast<const T*>(p + i);
    n = whole;
  }
  return (uint32_t)n;
}

// How the rows lie: every thread's units inside rows on 16-byte boundaries;
// rows on such boundaries with a ragged end; rows that start anywhere.
enum Rows { kFull, kEnds, kAnywhere };

// A unit from a staged row whose first byte lies `mis` bytes into it; `left`
// of the row's bytes begin at the unit (the columns past them are zero).
template <int DT, int ROWS>
__device__ __forceinline__ uint4 staged_unit(uint32_t at, uint32_t mis, int left) {
  uint4 r;
  if (ROWS != kAnywhere) {
    r = sm100::lds_u128(at);
  } else {
    const uint32_t p = at + (mis & ~3u);
    uint32_t w[5];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = sm100::lds_u32(p + 4 * i);
    if (elem_size(DT) == 2 && (mis & 2u)) {
      w[4] = sm100::lds_u32(p + 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (ROWS != kFull && left < 16) {
    uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (left <= 4 * i) w[i] = 0u;
      else if (left == 4 * i + 2) w[i] &= 0xFFFFu;
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}

// The warp's units, the first lane's first one being u0.
template <int DT, int ROWS, int K>
__device__ __forceinline__ void put_units(char* out, uint32_t u0, int64_t bytes,
                                          const uint4 (&r)[K]) {
  const bool inner =
      ROWS == kFull || (int64_t)u0 * 16 + K * 512 + (ROWS == kEnds ? 0 : 16) <= bytes;
  store_run<DT, ROWS != kAnywhere>(out, u0 * 16, inner, bytes, r);
}

// Sums of N (1 or 2) values over the row's warps, for the ring kernels: over
// a warp's lanes by shuffles, over the warps from shared memory, which every
// thread reads whole (fewer steps in a row than shuffles again).  `slot`
// holds zeros past the last warp.  The named barrier leaves the producer warp
// out, and carries whether a thread's wait ran out (then every thread leaves
// its row loop).
template <int N>
struct RowsSum {
  float (*slot)[36 * N];
  int threads;
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&v)[N], bool& ok) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float s = v[0];
    if (N == 2) {
      const bool up = lane & 1;
      const float send = up ? v[0] : v[N - 1], stay = up ? v[N - 1] : v[0];
      s = stay + __shfl_xor_sync(0xffffffffu, send, 1);
    }
#pragma unroll
    for (int k = N; k < 32; k <<= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (lane < N) slot[turn][warp * N + lane] = s;
    uint32_t bad = ok ? 0u : 1u;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred.aligned q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(bad)
        : "r"(bad), "r"(threads)
        : "memory");
    ok = bad == 0u;
    const float4* w = reinterpret_cast<const float4*>(slot[turn]);
    float2 t = make_float2(0.0f, 0.0f);
    const int quads = threads / 32 * N / 4;  // whole or not, what lies past them is zero
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) {
      const float4 f = w[i];
      t = __fadd2_rn(t, make_float2(f.x, f.y));
      t = __fadd2_rn(t, make_float2(f.z, f.w));
    }
    if (quads > 2 * N - 1)
      for (int i = 2 * N; i <= quads; ++i) {
        const float4 f = w[i];
        t = __fadd2_rn(t, make_float2(f.x, f.y));
        t = __fadd2_rn(t, make_float2(f.z, f.w));
      }
    turn ^= 1;
    if (N == 2) {
      v[0] = t.x;
      v[N - 1] = t.y;
    } else {
      v[0] = t.x + t.y;
    }
  }
};

struct RingPos {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++st == stages) {
      st = 0;
      ph ^= 1u;
    }
  }
};

__device__ __forceinline__ void ring_end(bool ok, uint32_t* status) {
  if (ok) return;
  atomicOr(status, kStatusWaitTimeout);
  // copies in flight land before the block's memory goes
  const long long t0 = clock64();
  while (clock64() - t0 < 2000000ll) {
  }
}

}  // namespace gc
