// gc_norm.cu -- layer norm: forward (the input kept in 8 bits in the same
// pass, if asked), backward from the input or from its checkpoint, and the
// reduction of the weight's and bias's gradients over the rows.
//
//   forward   mean = sum(x) / n,  rstd = 1 / sqrt(sum((x - mean)^2) / n + eps),
//             y = (x - mean) rstd gamma + beta
//   backward  n_j = (x_j - mean) rstd,  d_j = dy_j gamma_j,
//             dx_j = rstd (d_j - mean(d) - n_j mean(d n)),
//             dgamma_j = sum over rows of dy_j n_j,  dbeta_j = sum of dy_j
//
// A row lives in the registers of the threads that own it (one warp for
// narrow rows, one block for wide ones), so x is read once: the mean, then
// the centred sum of squares (no cancellation), then the output.  All sums
// are fp32.  The backward blocks walk over many rows and keep the column
// sums of their rows in registers; one partial per block goes to scratch and
// a second small grid adds the partials in block order, so equal inputs
// give equal bits whatever the number of rows.
#include <algorithm>

#include "gc_act8.cuh"

namespace gc {
namespace {

constexpr int kMaxParts = kNormMaxParts;  // partial rows of the column sums

struct NormArgs {
  const void* x;         // input (forward; backward without a checkpoint)
  const void* dy;
  void* out;             // y or dx
  const void *gamma, *beta;
  float *mean, *rstd;
  uint8_t *codes, *scales;
  float *dgamma, *dbeta;  // gradients, or NULL
  float* part;            // [parts][2][cols]
  int64_t rows, cols, ldx, lddy, ldout, codes_pitch, scales_pitch;
  float eps;
  int ptype, accumulate;
};

// Eight parameters from column c on; `fill` where there is no vector.
__device__ __forceinline__ void load_params(float v[8], const void* p, int ptype, int64_t c,
                                            int valid, float fill) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fill;
  } else if (ptype == GC_F32) {
    load_chunk<GC_F32, true>(v, static_cast<const float*>(p) + c, valid);
  } else if (ptype == GC_BF16) {
    load_chunk<GC_BF16, true>(v, static_cast<const __nv_bfloat16*>(p) + c, valid);
  } else {
    load_chunk<GC_F16, true>(v, static_cast<const __half*>(p) + c, valid);
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

__device__ __forceinline__ int chunk_valid(int64_t c, int64_t cols) {
  return (int)max((int64_t)0, min((int64_t)kChunk, cols - c));
}

// K chunks per thread: chunk i of a thread starts at column
// (thread + i * threads) * 8.  K == 0: rows wider than the registers hold;
// the row is read again (from L2) for each of its three passes.
template <int DT, int K, bool WARP, bool VEC>
__global__ void __launch_bounds__(WARP ? 256 : 1024) norm_forward_kernel(NormArgs a) {
  using T = typename Elem<DT>::T;
  __shared__ float2 slot[2][32];
  RowSum<WARP> sum{slot};
  const int nt = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int per_block = WARP ? blockDim.x / 32 : 1;
  const int64_t first = (int64_t)blockIdx.x * per_block + (WARP ? threadIdx.x >> 5 : 0);
  const float inv_n = 1.0f / (float)a.cols;
  const int loops = K ? K : (int)((a.codes_pitch / kChunk + nt - 1) / nt);

  for (int64_t row = first; row < a.rows; row += (int64_t)gridDim.x * per_block) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    float v[K ? K : 1][8];
    auto fetch = [&](int i) -> float* {
      const int64_t c = ((int64_t)t + (int64_t)i * nt) * kChunk;
      float* d = v[K ? i : 0];
      load_chunk<DT, VEC>(d, x + c, chunk_valid(c, a.cols));
      return d;
    };
    float s = 0.0f;
    if (K) {
#pragma unroll
      for (int i = 0; i < K; ++i) fetch(i);
    }
#pragma unroll
    for (int i = 0; i < (K ? K : loops); ++i) {
      const float* d = K ? v[i] : fetch(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += d[j];
    }
    const float mean = sum(s) * inv_n;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < (K ? K : loops); ++i) {
      const float* d = K ? v[i] : fetch(i);
      const int valid = chunk_valid(((int64_t)t + (int64_t)i * nt) * kChunk, a.cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = j < valid ? d[j] - mean : 0.0f;
        q = fmaf(e, e, q);
      }
    }
    const float rstd = rsqrtf(sum(q) * inv_n + a.eps);
    if (t == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < (K ? K : loops); ++i) {
      const float* d = K ? v[i] : fetch(i);
      const int64_t c = ((int64_t)t + (int64_t)i * nt) * kChunk;
      const int valid = chunk_valid(c, a.cols);
      if (a.codes) {
        const uint32_t b = scale_byte(group_max_bits(d));
        if (c < a.codes_pitch) {
          *reinterpret_cast<uint2*>(a.codes + row * a.codes_pitch + c) = encode8(d, b);
          if ((t & 3) == 0) a.scales[row * a.scales_pitch + c / kActGroup] = (uint8_t)b;
        }
      }
      if (valid > 0) {
        float g[8], bt[8], y[8];
        load_params(g, a.gamma, a.ptype, c, valid, 1.0f);
        load_params(bt, a.beta, a.ptype, c, valid, 0.0f);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = fmaf((d[j] - mean) * rstd, g[j], bt[j]);
        store_chunk<DT, VEC>(static_cast<T*>(a.out) + row * a.ldout + c, y, valid);
      }
    }
  }
}

template <int DT, bool CKPT, bool VEC>
__device__ __forceinline__ void load_input(float v[8], const NormArgs& a, int64_t row, int64_t c,
                                           int valid) {
  using T = typename Elem<DT>::T;
  if (CKPT) {
    const uint2 w =
        valid > 0 ? __ldg(reinterpret_cast<const uint2*>(a.codes + row * a.codes_pitch + c))
                  : make_uint2(0u, 0u);
    const uint32_t b = valid > 0 ? __ldg(a.scales + row * a.scales_pitch + c / kActGroup) : 0u;
    decode8(v, w, b);
  } else {
    load_chunk<DT, VEC>(v, static_cast<const T*>(a.x) + row * a.ldx + c, valid);
  }
}

// One row per block (or warp) at a time.  PARTS: also the column sums, kept
// in registers over the block's rows; K == 0 (wide rows) leaves them to
// norm_columns_kernel.
template <int DT, int K, bool WARP, bool CKPT, bool VEC>
__global__ void __launch_bounds__(WARP ? 256 : 512) norm_backward_kernel(NormArgs a) {
  using T = typename Elem<DT>::T;
  constexpr int KK = K ? K : 1;
  __shared__ float2 slot[2][32];
  RowSum<WARP> sum{slot};
  const int nt = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int per_block = WARP ? blockDim.x / 32 : 1;
  const int64_t first = (int64_t)blockIdx.x * per_block + (WARP ? threadIdx.x >> 5 : 0);
  const float inv_n = 1.0f / (float)a.cols;
  const int loops = K ? K : (int)((a.codes_pitch / kChunk + nt - 1) / nt);
  float sg[KK][8], sb[KK][8];
#pragma unroll
  for (int i = 0; i < KK; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sg[i][j] = sb[i][j] = 0.0f;

  for (int64_t row = first; row < a.rows; row += (int64_t)gridDim.x * per_block) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float d[KK][8], n[KK][8];
    float s1 = 0.0f, s2 = 0.0f;
    auto fetch = [&](int i) {  // d = dy gamma, n = (x - mean) rstd; the column sums
      const int64_t c = ((int64_t)t + (int64_t)i * nt) * kChunk;
      const int valid = chunk_valid(c, a.cols);
      const int k = K ? i : 0;
      float g[8];
      load_chunk<DT, VEC>(d[k], dy + c, valid);
      load_input<DT, CKPT, VEC>(n[k], a, row, c, valid);
      load_params(g, a.gamma, a.ptype, c, valid, 1.0f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[k][j] = (n[k][j] - mean) * rstd;
        if (K) {
          sg[k][j] = fmaf(d[k][j], n[k][j], sg[k][j]);
          sb[k][j] += d[k][j];
        }
        d[k][j] = j < valid ? d[k][j] * g[j] : 0.0f;
      }
    };
#pragma unroll
    for (int i = 0; i < (K ? K : loops); ++i) {
      fetch(i);
      const int k = K ? i : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s1 += d[k][j];
        s2 = fmaf(d[k][j], n[k][j], s2);
      }
    }
    const float2 c12 = sum(s1, s2);
    const float c1 = c12.x * inv_n, c2 = c12.y * inv_n;
#pragma unroll
    for (int i = 0; i < (K ? K : loops); ++i) {
      if (!K) fetch(i);
      const int k = K ? i : 0;
      const int64_t c = ((int64_t)t + (int64_t)i * nt) * kChunk;
      const int valid = chunk_valid(c, a.cols);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = rstd * (d[k][j] - c1 - n[k][j] * c2);
      if (valid > 0) store_chunk<DT, VEC>(static_cast<T*>(a.out) + row * a.ldout + c, o, valid);
    }
  }

  if (K == 0) return;
  if (!a.dgamma && !a.dbeta) return;
  // the block's warps own the same columns when a row is one warp's: add
  // them in warp order
  extern __shared__ float acc[];  // WARP: [2][cols padded to 8]
  float* pg = a.part + (int64_t)blockIdx.x * 2 * a.cols;
  float* pb = pg + a.cols;
  if (WARP) {
    const int w8 = (int)a.codes_pitch;
    for (int w = 0; w < per_block; ++w) {
      if ((int)(threadIdx.x >> 5) == w) {
#pragma unroll
        for (int i = 0; i < KK; ++i) {
          const int c = (t + i * 32) * kChunk;
          if (c < w8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              acc[c + j] = (w ? acc[c + j] : 0.0f) + sg[i][j];
              acc[w8 + c + j] = (w ? acc[w8 + c + j] : 0.0f) + sb[i][j];
            }
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      pg[c] = acc[c];
      pb[c] = acc[w8 + c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < KK; ++i) {
      const int64_t c = ((int64_t)t + (int64_t)i * nt) * kChunk;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < a.cols) {
          pg[c + j] = sg[i][j];
          pb[c + j] = sb[i][j];
        }
    }
  }
}

// Column sums of wide rows: block (x, y) adds rows y, y + gridDim.y, ... of
// 8 * 256 columns into partial row y.
template <int DT, bool CKPT, bool VEC>
__global__ void __launch_bounds__(256) norm_columns_kernel(NormArgs a) {
  using T = typename Elem<DT>::T;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * kChunk;
  const int valid = chunk_valid(c, a.cols);
  if (valid <= 0) return;
  float sg[8] = {}, sb[8] = {};
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float d[8], n[8];
    load_chunk<DT, VEC>(d, static_cast<const T*>(a.dy) + row * a.lddy + c, valid);
    load_input<DT, CKPT, VEC>(n, a, row, c, valid);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sg[j] = fmaf(d[j], (n[j] - mean) * rstd, sg[j]);
      sb[j] += d[j];
    }
  }
  float* pg = a.part + (int64_t)blockIdx.y * 2 * a.cols;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < valid) {
      pg[c + j] = sg[j];
      pg[a.cols + c + j] = sb[j];
    }
}

// out[c] (+)= the sum of part[p][which][c] over p in order: a block takes 32
// columns of one of the two sums; its 16 warps add every 16th partial row,
// then the warps' sums are added in warp order.
__global__ void __launch_bounds__(512) norm_reduce_kernel(const float* part, int parts,
                                                          int64_t cols, float* dgamma,
                                                          float* dbeta, int accumulate) {
  __shared__ float s[16][33];
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < cols)
    for (int p = warp; p < parts; p += 16)
      v += part[((int64_t)p * 2 + blockIdx.y) * cols + c];
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < cols) {
    v = s[0][lane];
#pragma unroll
    for (int w = 1; w < 16; ++w) v += s[w][lane];
    out[c] = accumulate ? out[c] + v : v;
  }
}

int elem_size(int dtype) { return dtype == GC_F32 ? 4 : 2; }
bool row_aligned(int64_t ld, int dtype) { return ld * elem_size(dtype) % 16 == 0; }

// How a row is spread: K chunks for each of `threads` threads.
struct RowPlan {
  int k, threads;  // k == 0: wider than the registers hold
  bool warp;
};

RowPlan row_plan(int64_t cols, int max_threads) {
  const int64_t chunks = ckpt_codes_pitch(cols) / kChunk;
  if (chunks <= 32 * 4) return {(int)ceil_div(chunks, 32), 256, true};
  for (int k = 1; k <= 4; ++k) {
    const int64_t t = round_up(ceil_div(chunks, k), 32);
    if (t <= (k < 4 ? std::min(256 * k, max_threads) : max_threads)) return {k, (int)t, false};
  }
  return {0, max_threads, false};
}

template <int DT, int K, bool WARP>
void forward_launch(gc_ctx* ctx, const NormArgs& a, unsigned grid, int threads, bool vec) {
  if (vec)
    norm_forward_kernel<DT, K, WARP, true><<<grid, threads, 0, ctx->stream>>>(a);
  else
    norm_forward_kernel<DT, K, WARP, false><<<grid, threads, 0, ctx->stream>>>(a);
}

template <int DT>
void forward_dt(gc_ctx* ctx, const NormArgs& a, bool vec) {
  const RowPlan p = row_plan(a.cols, 1024);
  const int64_t blocks = p.warp ? ceil_div(a.rows, (int64_t)(p.threads / 32)) : a.rows;
  const unsigned g = (unsigned)std::min<int64_t>(
      blocks, (int64_t)ctx->num_sms * std::max(1, 2048 / p.threads));
  if (p.warp) {
    if (p.k == 1) forward_launch<DT, 1, true>(ctx, a, g, p.threads, vec);
    else if (p.k == 2) forward_launch<DT, 2, true>(ctx, a, g, p.threads, vec);
    else if (p.k == 3) forward_launch<DT, 3, true>(ctx, a, g, p.threads, vec);
    else forward_launch<DT, 4, true>(ctx, a, g, p.threads, vec);
  } else {
    if (p.k == 1) forward_launch<DT, 1, false>(ctx, a, g, p.threads, vec);
    else if (p.k == 2) forward_launch<DT, 2, false>(ctx, a, g, p.threads, vec);
    else if (p.k == 3) forward_launch<DT, 3, false>(ctx, a, g, p.threads, vec);
    else if (p.k == 4) forward_launch<DT, 4, false>(ctx, a, g, p.threads, vec);
    else forward_launch<DT, 0, false>(ctx, a, g, p.threads, vec);
  }
}

template <int DT, int K, bool WARP, bool CKPT>
void backward_launch(gc_ctx* ctx, const NormArgs& a, unsigned grid, int threads, bool vec) {
  const size_t smem = WARP ? (size_t)a.codes_pitch * 2 * sizeof(float) : 0;
  if (vec)
    norm_backward_kernel<DT, K, WARP, CKPT, true><<<grid, threads, smem, ctx->stream>>>(a);
  else
    norm_backward_kernel<DT, K, WARP, CKPT, false><<<grid, threads, smem, ctx->stream>>>(a);
}

template <int DT, bool CKPT>
int backward_dt(gc_ctx* ctx, const NormArgs& a, bool vec) {
  const RowPlan p = row_plan(a.cols, 512);
  const int64_t blocks = p.warp ? ceil_div(a.rows, (int64_t)(p.threads / 32)) : a.rows;
  const int64_t cap = p.k ? std::min<int64_t>((int64_t)ctx->num_sms * 2, kMaxParts)
                          : (int64_t)ctx->num_sms * 4;
  const unsigned g = (unsigned)std::min<int64_t>(blocks, cap);
  if (p.warp) {
    if (p.k == 1) backward_launch<DT, 1, true, CKPT>(ctx, a, g, p.threads, vec);
    else if (p.k == 2) backward_launch<DT, 2, true, CKPT>(ctx, a, g, p.threads, vec);
    else if (p.k == 3) backward_launch<DT, 3, true, CKPT>(ctx, a, g, p.threads, vec);
    else backward_launch<DT, 4, true, CKPT>(ctx, a, g, p.threads, vec);
    return (int)g;
  }
  if (p.k == 1) backward_launch<DT, 1, false, CKPT>(ctx, a, g, p.threads, vec);
  else if (p.k == 2) backward_launch<DT, 2, false, CKPT>(ctx, a, g, p.threads, vec);
  else if (p.k == 3) backward_launch<DT, 3, false, CKPT>(ctx, a, g, p.threads, vec);
  else if (p.k == 4) backward_launch<DT, 4, false, CKPT>(ctx, a, g, p.threads, vec);
  else backward_launch<DT, 0, false, CKPT>(ctx, a, g, p.threads, vec);
  return p.k ? (int)g : 0;
}

template <int DT, bool CKPT>
int columns_dt(gc_ctx* ctx, const NormArgs& a, bool vec) {
  const int64_t bx = ceil_div(ceil_div(a.cols, (int64_t)kChunk), 256);
  const int64_t by = std::max<int64_t>(
      1, std::min<int64_t>({ceil_div(a.rows, 16), (int64_t)kMaxParts,
                            ceil_div((int64_t)ctx->num_sms * 8, bx)}));
  const dim3 g((unsigned)bx, (unsigned)by);
  if (vec)
    norm_columns_kernel<DT, CKPT, true><<<g, 256, 0, ctx->stream>>>(a);
  else
    norm_columns_kernel<DT, CKPT, false><<<g, 256, 0, ctx->stream>>>(a);
  return (int)by;
}

template <int DT>
gc_status backward_all(gc_ctx* ctx, const NormArgs& a, bool vec) {
  int parts = 0;
  if (a.rows > 0) {
    {
      LaunchScope L(ctx, GC_PHASE_NORM_BACKWARD);
      parts = a.codes ? backward_dt<DT, true>(ctx, a, vec) : backward_dt<DT, false>(ctx, a, vec);
    }
    if (parts == 0 && (a.dgamma || a.dbeta)) {
      LaunchScope L(ctx, GC_PHASE_NORM_BACKWARD);
      parts = a.codes ? columns_dt<DT, true>(ctx, a, vec) : columns_dt<DT, false>(ctx, a, vec);
    }
  }
  if (a.dgamma || a.dbeta) {
    LaunchScope L(ctx, GC_PHASE_NORM_REDUCE);
    norm_reduce_kernel<<<dim3((unsigned)ceil_div(a.cols, 32), 2), 512, 0, ctx->stream>>>(
        a.part, parts, a.cols, a.dgamma, a.dbeta, a.accumulate);
  }
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

}  // namespace

int64_t norm_scratch_bytes(int64_t rows, int64_t cols) {
  return std::min<int64_t>(std::max<int64_t>(rows, 1), kMaxParts) * 2 * cols * (int64_t)sizeof(float);
}

gc_status launch_norm_forward(gc_ctx* ctx, const void* x, int dtype, int64_t rows, int64_t cols,
                              int64_t ldx, const void* gamma, const void* beta, int ptype,
                              float eps, void* y, int64_t ldy, float* mean, float* rstd,
                              uint8_t* codes, uint8_t* scales) {
  if (rows == 0 || cols == 0) return GC_OK;
  NormArgs a{};
  a.x = x;
  a.out = y;
  a.gamma = gamma;
  a.beta = beta;
  a.mean = mean;
  a.rstd = rstd;
  a.codes = codes;
  a.scales = scales;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.ldout = ldy;
  a.codes_pitch = ckpt_codes_pitch(cols);
  a.scales_pitch = ckpt_scales_pitch(cols);
  a.eps = eps;
  a.ptype = ptype;
  const bool vec = row_aligned(ldx, dtype) && row_aligned(ldy, dtype);
  LaunchScope L(ctx, GC_PHASE_NORM_FORWARD);
  if (dtype == GC_F32) forward_dt<GC_F32>(ctx, a, vec);
  else if (dtype == GC_BF16) forward_dt<GC_BF16>(ctx, a, vec);
  else forward_dt<GC_F16>(ctx, a, vec);
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

gc_status launch_norm_backward(gc_ctx* ctx, const void* dy, int64_t lddy, const void* x,
                               int64_t ldx, const uint8_t* codes, const uint8_t* scales, int dtype,
                               int64_t rows, int64_t cols, const void* gamma, int ptype,
                               const float* mean, const float* rstd, void* dx, int64_t lddx,
                               float* dgamma, float* dbeta, int accumulate, float* part) {
  if (cols == 0) return GC_OK;
  NormArgs a{};
  a.x = x;
  a.dy = dy;
  a.out = dx;
  a.gamma = gamma;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.part = part;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.lddy = lddy;
  a.ldout = lddx;
  a.codes_pitch = ckpt_codes_pitch(cols);
  a.scales_pitch = ckpt_scales_pitch(cols);
  a.ptype = ptype;
  a.accumulate = accumulate;
  const bool vec = row_aligned(lddy, dtype) && row_aligned(lddx, dtype) &&
                   (codes || row_aligned(ldx, dtype));
  if (dtype == GC_F32) return backward_all<GC_F32>(ctx, a, vec);
  if (dtype == GC_BF16) return backward_all<GC_BF16>(ctx, a, vec);
  return backward_all<GC_F16>(ctx, a, vec);
}

}  // namespace gc
