// gc_wgrad.cu -- the weight and bias gradients of a linear layer from the
// output's gradient and the 8-bit checkpoint of its input:
//
//   dw[o][i] (+)= sum over tokens t of dy[t][o] x^[t][i]
//   db[o]    (+)= sum over tokens t of dy[t][o]
#include <algorithm>

#include "gc_act8.cuh"

namespace gc {
namespace {

constexpr int kTile = 64;   // outputs and inputs of a block's tile
constexpr int kStep = 16;   // tokens per step

struct WgradArgs {
  const void* dy;
  const uint8_t *codes, *scales;
  float *dw, *db;
  int64_t rows, out, in, lddy, lddw, codes_pitch, scales_pitch;
  int accumulate;
};

template <int DT>
__global__ void __launch_bounds__(256) wgrad_kernel(WgradArgs a) {
  using E = Elem<DT>;
  __shared__ float sd[kStep][kTile], sx[kStep][kTile];
  const int64_t o0 = (int64_t)blockIdx.y * kTile, i0 = (int64_t)blockIdx.x * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {}, bias[4] = {};
  for (int64_t t0 = 0; t0 < a.rows; t0 += kStep) {
    for (int e = threadIdx.x; e < kStep * kTile; e += 256) {
      const int r = e / kTile, c = e % kTile;
      const int64_t t = t0 + r;
      float d = 0.0f, x = 0.0f;
      if (t < a.rows && o0 + c < a.out)
        d = E::to_float(static_cast<const typename E::T*>(a.dy)[t * a.lddy + o0 + c]);
      if (t < a.rows && i0 + c < a.in)
        x = decode1(a.codes[t * a.codes_pitch + i0 + c], 0,
                    (uint32_t)a.scales[t * a.scales_pitch + (i0 + c) / kActGroup] << 23);
      sd[r][c] = d;
      sx[r][c] = x;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kStep; ++r) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float d = sd[r][ty * 4 + p];
        bias[p] += d;
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[p][q] = fmaf(d, sx[r][tx * 4 + q], acc[p][q]);
      }
    }
    __syncthreads();
  }
  for (int p = 0; p < 4; ++p) {
    const int64_t o = o0 + ty * 4 + p;
    if (o >= a.out) continue;
    for (int q = 0; q < 4; ++q) {
      const int64_t i = i0 + tx * 4 + q;
      if (i >= a.in) continue;
      float* w = a.dw + o * a.lddw + i;
      *w = a.accumulate ? *w + acc[p][q] : acc[p][q];
    }
    if (a.db && blockIdx.x == 0 && tx == 0)
      a.db[o] = a.accumulate ? a.db[o] + bias[p] : bias[p];
  }
}

}  // namespace

int64_t wgrad_scratch_bytes(int64_t rows, int64_t out, int64_t in, int dtype) { return 0; }

gc_status launch_wgrad(gc_ctx* ctx, const void* dy, int dtype, int64_t lddy, const uint8_t* codes,
                       const uint8_t* scales, int64_t rows, int64_t out, int64_t in, float* dw,
                       int64_t lddw, float* db, int accumulate, void* scratch) {
  if (out == 0 || in == 0) return GC_OK;
  WgradArgs a{};
  a.dy = dy;
  a.codes = codes;
  a.scales = scales;
  a.dw = dw;
  a.db = db;
  a.rows = rows;
  a.out = out;
  a.in = in;
  a.lddy = lddy;
  a.lddw = lddw;
  a.codes_pitch = ckpt_codes_pitch(in);
  a.scales_pitch = ckpt_scales_pitch(in);
  a.accumulate = accumulate;
  LaunchScope L(ctx, GC_PHASE_WGRAD);
  const dim3 g((unsigned)ceil_div(in, kTile), (unsigned)ceil_div(out, kTile));
  if (dtype == GC_F32) wgrad_kernel<GC_F32><<<g, 256, 0, ctx->stream>>>(a);
  else if (dtype == GC_BF16) wgrad_kernel<GC_BF16><<<g, 256, 0, ctx->stream>>>(a);
  else wgrad_kernel<GC_F16><<<g, 256, 0, ctx->stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

}  // namespace gc
