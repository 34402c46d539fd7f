// gc_rows.cuh -- what the kernels that walk over rows share (gc_norm.cu,
// gc_rms.cu): parameters per column and sums over the threads of a row.
#pragma once

#include "gc_act8.cuh"

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

}  // namespace gc
