// gc_ckpt.cu -- activations kept in 8 bits, and the activation functions
// around them: save and restore, y = f(x) [* gate] with the inputs saved in
// the same pass, and the backward pass from the saved inputs.
//
//   GELU: f(x) = x Phi(x),  f'(x) = Phi(x) + x phi(x)
//   SiLU: f(x) = x s(x),    f'(x) = s(x) (1 + x (1 - s(x)))
//   backward: dx = dy [* gate^] f'(x^), dgate = dy f(x^), with x^ and gate^
//   the values that the checkpoints stand for.
//
// Every kernel is one pass over its tensors, bound by memory: a thread owns a
// chunk of 8 consecutive columns (one 16-byte load per 16-bit tensor), four
// neighbouring threads the group of 32 that shares a scale byte.  The chunks
// of all rows are one index space, so that narrow and wide rows load the GPU
// alike.
#include <algorithm>

#include "gc_act8.cuh"

namespace gc {
namespace {

constexpr int kThreads = 256;
constexpr int kKindNone = 2;  // save only

// Position of a thread in the (row, chunk) space, advanced by a fixed stride
// without a division per step.
struct Walk {
  int64_t row;
  int32_t chunk;
  int64_t step_rows;
  int32_t step_chunks, per_row;
  __device__ __forceinline__ Walk(int64_t first, int64_t stride, int32_t chunks_per_row)
      : per_row(chunks_per_row) {
    row = first / per_row;
    chunk = (int32_t)(first - row * per_row);
    step_rows = stride / per_row;
    step_chunks = (int32_t)(stride - step_rows * per_row);
  }
  __device__ __forceinline__ void next() {
    row += step_rows;
    chunk += step_chunks;
    if (chunk >= per_row) {
      chunk -= per_row;
      ++row;
    }
  }
};

template <int KIND>
__device__ __forceinline__ float act_value(float x) {
  if (KIND == GC_GELU) return 0.5f * x * (1.0f + erff(x * 0.70710678f));
  return x / (1.0f + expf(-x));
}

// f(x) and f'(x).
template <int KIND>
__device__ __forceinline__ void act_both(float x, float& f, float& d) {
  if (KIND == GC_GELU) {
    const float cdf = 0.5f * (1.0f + erff(x * 0.70710678f));
    f = x * cdf;
    d = fmaf(x * 0.39894228f, expf(-0.5f * x * x), cdf);
  } else {
    const float s = 1.0f / (1.0f + expf(-x));
    f = x * s;
    d = s * fmaf(x, 1.0f - s, 1.0f);
  }
}

struct FwdArgs {
  const void* x;
  const void* gate;
  void* y;
  uint8_t *codes, *scales, *gate_codes, *gate_scales;
  int64_t ldx, ldgate, ldy;
  int64_t total;  // chunks of all rows
  int64_t cols, codes_pitch, scales_pitch;
};

template <int DT, int KIND, bool GATED, bool VEC>
__global__ void __launch_bounds__(kThreads) act_forward_kernel(FwdArgs a) {
  using T = typename Elem<DT>::T;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  Walk w(first, stride, (int32_t)(a.codes_pitch / kChunk));
  // whole warps stay in the loop together (group_max_bits); a.total is a
  // multiple of 4, so a group of 32 columns is wholly inside or outside
  for (int64_t base = first - (threadIdx.x & 31); base < a.total; base += stride, w.next()) {
    const bool in = base + (threadIdx.x & 31) < a.total;
    const int64_t c = (int64_t)w.chunk * kChunk;
    const int valid = in ? (int)max((int64_t)0, min((int64_t)kChunk, a.cols - c)) : 0;
    float v[8], g[8];
    load_chunk<DT, VEC>(v, static_cast<const T*>(a.x) + w.row * a.ldx + c, valid);
    if (GATED) load_chunk<DT, VEC>(g, static_cast<const T*>(a.gate) + w.row * a.ldgate + c, valid);
    if (KIND != kKindNone) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = act_value<KIND>(v[i]);
        if (GATED) y[i] *= g[i];
      }
      store_chunk<DT, VEC>(static_cast<T*>(a.y) + w.row * a.ldy + c, y, valid);
    }
    if (a.codes) {
      const uint32_t b = scale_byte(group_max_bits(v));
      const uint32_t bg = GATED ? scale_byte(group_max_bits(g)) : 0u;
      if (in) {
        const int64_t at = w.row * a.codes_pitch + c;
        *reinterpret_cast<uint2*>(a.codes + at) = encode8(v, b);
        if (GATED) *reinterpret_cast<uint2*>(a.gate_codes + at) = encode8(g, bg);
        if ((w.chunk & 3) == 0) {
          const int64_t sat = w.row * a.scales_pitch + (w.chunk >> 2);
          a.scales[sat] = (uint8_t)b;
          if (GATED) a.gate_scales[sat] = (uint8_t)bg;
        }
      }
    }
  }
}

struct BwdArgs {
  const void* dy;
  void *dx, *dgate;
  const uint8_t *codes, *scales, *gate_codes, *gate_scales;
  int64_t lddy, lddx, lddgate;
  int64_t total, cols, codes_pitch, scales_pitch;
};

__device__ __forceinline__ void restore_chunk(float v[8], const uint8_t* codes,
                                              const uint8_t* scales, int64_t row, int32_t chunk,
                                              int64_t cp, int64_t sp) {
  const uint2 c = __ldg(reinterpret_cast<const uint2*>(codes + row * cp + (int64_t)chunk * kChunk));
  decode8(v, c, __ldg(scales + row * sp + (chunk >> 2)));
}

template <int DT, int KIND, bool GATED, bool VEC>
__global__ void __launch_bounds__(kThreads) act_backward_kernel(BwdArgs a) {
  using T = typename Elem<DT>::T;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  Walk w(first, stride, (int32_t)(a.codes_pitch / kChunk));
  for (int64_t at = first; at < a.total; at += stride, w.next()) {
    const int64_t c = (int64_t)w.chunk * kChunk;
    const int valid = (int)min((int64_t)kChunk, a.cols - c);
    if (valid <= 0) continue;
    float dy[8], x[8], g[8];
    load_chunk<DT, VEC>(dy, static_cast<const T*>(a.dy) + w.row * a.lddy + c, valid);
    restore_chunk(x, a.codes, a.scales, w.row, w.chunk, a.codes_pitch, a.scales_pitch);
    if (GATED)
      restore_chunk(g, a.gate_codes, a.gate_scales, w.row, w.chunk, a.codes_pitch,
                    a.scales_pitch);
    float dx[8], dg[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f, d;
      act_both<KIND>(x[i], f, d);
      dx[i] = GATED ? dy[i] * g[i] * d : dy[i] * d;
      dg[i] = dy[i] * f;
    }
    store_chunk<DT, VEC>(static_cast<T*>(a.dx) + w.row * a.lddx + c, dx, valid);
    if (GATED) store_chunk<DT, VEC>(static_cast<T*>(a.dgate) + w.row * a.lddgate + c, dg, valid);
  }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) restore_kernel(BwdArgs a) {
  using T = typename Elem<DT>::T;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  Walk w(first, stride, (int32_t)(a.codes_pitch / kChunk));
  for (int64_t at = first; at < a.total; at += stride, w.next()) {
    const int64_t c = (int64_t)w.chunk * kChunk;
    const int valid = (int)min((int64_t)kChunk, a.cols - c);
    if (valid <= 0) continue;
    float x[8];
    restore_chunk(x, a.codes, a.scales, w.row, w.chunk, a.codes_pitch, a.scales_pitch);
    store_chunk<DT, VEC>(static_cast<T*>(a.dx) + w.row * a.lddx + c, x, valid);
  }
}

int elem_size(int dtype) { return dtype == GC_F32 ? 4 : 2; }

unsigned grid_for(const gc_ctx* ctx, int64_t total) {
  return (unsigned)std::max<int64_t>(
      1, std::min<int64_t>(ceil_div(total, kThreads), (int64_t)ctx->num_sms * 8));
}

template <int DT, int KIND, bool GATED>
void forward_dt(gc_ctx* ctx, const FwdArgs& a, bool vec) {
  const unsigned g = grid_for(ctx, a.total);
  if (vec)
    act_forward_kernel<DT, KIND, GATED, true><<<g, kThreads, 0, ctx->stream>>>(a);
  else
    act_forward_kernel<DT, KIND, GATED, false><<<g, kThreads, 0, ctx->stream>>>(a);
}

template <int KIND, bool GATED>
void forward_kind(gc_ctx* ctx, const FwdArgs& a, int dtype, bool vec) {
  if (dtype == GC_F32) forward_dt<GC_F32, KIND, GATED>(ctx, a, vec);
  else if (dtype == GC_BF16) forward_dt<GC_BF16, KIND, GATED>(ctx, a, vec);
  else forward_dt<GC_F16, KIND, GATED>(ctx, a, vec);
}

template <int DT, int KIND, bool GATED>
void backward_dt(gc_ctx* ctx, const BwdArgs& a, bool vec) {
  const unsigned g = grid_for(ctx, a.total);
  if (vec)
    act_backward_kernel<DT, KIND, GATED, true><<<g, kThreads, 0, ctx->stream>>>(a);
  else
    act_backward_kernel<DT, KIND, GATED, false><<<g, kThreads, 0, ctx->stream>>>(a);
}

template <int KIND, bool GATED>
void backward_kind(gc_ctx* ctx, const BwdArgs& a, int dtype, bool vec) {
  if (dtype == GC_F32) backward_dt<GC_F32, KIND, GATED>(ctx, a, vec);
  else if (dtype == GC_BF16) backward_dt<GC_BF16, KIND, GATED>(ctx, a, vec);
  else backward_dt<GC_F16, KIND, GATED>(ctx, a, vec);
}

template <int DT>
void restore_dt(gc_ctx* ctx, const BwdArgs& a, bool vec) {
  const unsigned g = grid_for(ctx, a.total);
  if (vec)
    restore_kernel<DT, true><<<g, kThreads, 0, ctx->stream>>>(a);
  else
    restore_kernel<DT, false><<<g, kThreads, 0, ctx->stream>>>(a);
}

bool row_aligned(int64_t ld, int dtype) { return ld * elem_size(dtype) % 16 == 0; }

gc_status launched() { return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA; }

}  // namespace

gc_status launch_ckpt_save(gc_ctx* ctx, const void* x, int dtype, int64_t rows, int64_t cols,
                           int64_t ldx, uint8_t* codes, uint8_t* scales) {
  if (rows == 0 || cols == 0) return GC_OK;
  FwdArgs a{};
  a.x = x;
  a.codes = codes;
  a.scales = scales;
  a.ldx = ldx;
  a.cols = cols;
  a.codes_pitch = ckpt_codes_pitch(cols);
  a.scales_pitch = ckpt_scales_pitch(cols);
  a.total = rows * (a.codes_pitch / kChunk);
  LaunchScope L(ctx, GC_PHASE_CKPT_SAVE);
  forward_kind<kKindNone, false>(ctx, a, dtype, row_aligned(ldx, dtype));
  return launched();
}

gc_status launch_ckpt_restore(gc_ctx* ctx, const uint8_t* codes, const uint8_t* scales, int dtype,
                              int64_t rows, int64_t cols, void* x_out, int64_t ldx) {
  if (rows == 0 || cols == 0) return GC_OK;
  BwdArgs a{};
  a.codes = codes;
  a.scales = scales;
  a.dx = x_out;
  a.lddx = ldx;
  a.cols = cols;
  a.codes_pitch = ckpt_codes_pitch(cols);
  a.scales_pitch = ckpt_scales_pitch(cols);
  a.total = rows * (a.codes_pitch / kChunk);
  const bool vec = row_aligned(ldx, dtype);
  LaunchScope L(ctx, GC_PHASE_CKPT_RESTORE);
  if (dtype == GC_F32) restore_dt<GC_F32>(ctx, a, vec);
  else if (dtype == GC_BF16) restore_dt<GC_BF16>(ctx, a, vec);
  else restore_dt<GC_F16>(ctx, a, vec);
  return launched();
}

gc_status launch_act_forward(gc_ctx* ctx, int kind, const void* x, int64_t ldx, const void* gate,
                             int64_t ldgate, int dtype, int64_t rows, int64_t cols, void* y,
                             int64_t ldy, uint8_t* codes, uint8_t* scales, uint8_t* gate_codes,
                             uint8_t* gate_scales) {
  if (rows == 0 || cols == 0) return GC_OK;
  FwdArgs a{};
  a.x = x;
  a.gate = gate;
  a.y = y;
  a.codes = codes;
  a.scales = scales;
  a.gate_codes = gate_codes;
  a.gate_scales = gate_scales;
  a.ldx = ldx;
  a.ldgate = ldgate;
  a.ldy = ldy;
  a.cols = cols;
  a.codes_pitch = ckpt_codes_pitch(cols);
  a.scales_pitch = ckpt_scales_pitch(cols);
  a.total = rows * (a.codes_pitch / kChunk);
  const bool vec = row_aligned(ldx, dtype) && row_aligned(ldy, dtype) &&
                   (!gate || row_aligned(ldgate, dtype));
  LaunchScope L(ctx, GC_PHASE_ACT_FORWARD);
  if (kind == GC_GELU) {
    if (gate) forward_kind<GC_GELU, true>(ctx, a, dtype, vec);
    else forward_kind<GC_GELU, false>(ctx, a, dtype, vec);
  } else {
    if (gate) forward_kind<GC_SILU, true>(ctx, a, dtype, vec);
    else forward_kind<GC_SILU, false>(ctx, a, dtype, vec);
  }
  return launched();
}

gc_status launch_act_backward(gc_ctx* ctx, int kind, const void* dy, int64_t lddy,
                              const uint8_t* codes, const uint8_t* scales,
                              const uint8_t* gate_codes, const uint8_t* gate_scales, int dtype,
                              int64_t rows, int64_t cols, void* dx, int64_t lddx, void* dgate,
                              int64_t lddgate) {
  if (rows == 0 || cols == 0) return GC_OK;
  BwdArgs a{};
  a.dy = dy;
  a.dx = dx;
  a.dgate = dgate;
  a.codes = codes;
  a.scales = scales;
  a.gate_codes = gate_codes;
  a.gate_scales = gate_scales;
  a.lddy = lddy;
  a.lddx = lddx;
  a.lddgate = lddgate;
  a.cols = cols;
  a.codes_pitch = ckpt_codes_pitch(cols);
  a.scales_pitch = ckpt_scales_pitch(cols);
  a.total = rows * (a.codes_pitch / kChunk);
  const bool vec = row_aligned(lddy, dtype) && row_aligned(lddx, dtype) &&
                   (!dgate || row_aligned(lddgate, dtype));
  LaunchScope L(ctx, GC_PHASE_ACT_BACKWARD);
  if (kind == GC_GELU) {
    if (dgate) backward_kind<GC_GELU, true>(ctx, a, dtype, vec);
    else backward_kind<GC_GELU, false>(ctx, a, dtype, vec);
  } else {
    if (dgate) backward_kind<GC_SILU, true>(ctx, a, dtype, vec);
    else backward_kind<GC_SILU, false>(ctx, a, dtype, vec);
  }
  return launched();
}

}  // namespace gc
