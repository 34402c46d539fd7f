// gc_ckpt.cu -- activations kept in 8 bits, and the activation functions
// around them: save and restore, y = f(x) [* gate] with the inputs saved in
// the same pass, and the backward pass from the saved inputs.
//
//   GELU: f(x) = x Phi(x),  f'(x) = Phi(x) + x phi(x)
//   SiLU: f(x) = x s(x),    f'(x) = s(x) (1 + x (1 - s(x)))
//   backward: dx = dy [* gate^] f'(x^), dgate = dy f(x^), with x^ and gate^
//   the values that the checkpoints stand for.
//
// Every kernel is one pass over its tensors, bound by memory as long as few
// instructions are spent per element.  A warp takes a run of U x 32
// consecutive units of 16 bytes of one row: it divides once, adds constants
// to one base address per tensor, and issues all its loads before it uses
// the first.  (A thread that placed each of its units by itself spent 40
// instructions per element on a gated forward pass, half of them on
// addresses: 138 us for 8192 x 11008 bf16 against 107 at the copy rate.)
// Rows that do not start on 16-byte boundaries are read and written in the
// aligned pieces that cover the run, shifted into place between lanes.
//
// Measured, bytes read and written once over the time (a plain copy: 6.77
// TB/s): gated SiLU 8192 x 11008 bf16 forward 113 us (6.4 TB/s), backward 131
// (5.5); save and restore 8192 x 4096 fp32 58 us one after the other (5.8),
// 16384 x 4096 bf16 34 and 35 (6.0, 5.8); GELU 8192 x 4096 fp16 33 and 40,
// fp32 47 and 58.  Unaligned rows spend instructions on the shifting of every
// unit: GELU 4093 x 4097 fp16 27 and 27 us (3.1 and 3.2 TB/s) at 81% and 73%
// of the issue slots, SiLU 23 and 22.
#include <algorithm>

#include "gc_act8.cuh"

namespace gc {
namespace {

constexpr int kThreads = 256;
constexpr int kKindNone = 2;  // save, restore

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// f and, if asked, f' of two values: the passes come near the instruction
// rate, and the packed fp32 instructions take half the slots.
//
// GELU: with a = |x|, Phi(-a) = exp(-a^2 / 2) R(a), where R(a) =
// exp(a^2 / 2) Phi(-a) is smooth: a polynomial in t = 1 / (1 + c a), fitted on
// [0, 13.4] by iteratively reweighted least squares, so that Phi(-a) is off by
// little absolutely and as a part of itself.  The negative tail, where the
// function is x Phi(-a) alone, then keeps its digits down to where it leaves
// binary32's normal range (x = -13.1).  fp32: degree 7, 3.3e-8 / max(1, a) and
// 7.3e-7 of itself.  16-bit types: degree 6, 3.5e-8 / max(1, a) and 2^-14 of
// itself (an eighth of a half's rounding; a degree less is a packed instruction
// for two values, of about 46).  (Degree 5 for all, with the absolute error
// alone in the fit, was off by 1e-4 of the value at -5 and by 1e-2 at -12,
// more than a bf16 rounding.)  fp32 arithmetic adds the exponent's rounding,
// x^2 2^-23 of the tail.
//
// SiLU: s(x) = 2^-8 / (2^-8 + 2^-8 exp(-x)).  The factor keeps the reciprocal
// in the normal range as far down as x s(x) is in it (x = -91.8): the
// approximate instructions give 0 for what lies below.  fp16 has no such
// values (its least is 2^-24) and goes without.
template <int DT, int KIND, bool DERIV>
__device__ __forceinline__ void act(const float2& x, float2& f, float2& d) {
  if (KIND == GC_GELU) {
    const float2 a = make_float2(fabsf(x.x), fabsf(x.y));
    const float2 u = __ffma2_rn(a, both(DT == GC_F32 ? 0.34f : 0.28f), both(1.0f));
    const float2 t = make_float2(rcp_approx(u.x), rcp_approx(u.y));
    float2 r;
    if (DT == GC_F32) {
      r = __ffma2_rn(t, both(0.0472440794f), both(-0.211599767f));
      r = __ffma2_rn(r, t, both(0.285200179f));
      r = __ffma2_rn(r, t, both(-0.0523733199f));
      r = __ffma2_rn(r, t, both(0.169367765f));
      r = __ffma2_rn(r, t, both(0.125428692f));
      r = __ffma2_rn(r, t, both(0.136785954f));
      r = __ffma2_rn(r, t, both(-5.35652689e-05f));
    } else {
      r = __ffma2_rn(t, both(-0.108482867f), both(0.403031647f));
      r = __ffma2_rn(r, t, both(-0.263652384f));
      r = __ffma2_rn(r, t, both(0.297365874f));
      r = __ffma2_rn(r, t, both(0.0506336838f));
      r = __ffma2_rn(r, t, both(0.121776283f));
      r = __ffma2_rn(r, t, both(-0.000672220427f));
    }
    const float2 v = __fmul2_rn(__fmul2_rn(a, a), both(-0.72134752f));
    const float2 e = make_float2(exp2_approx(v.x), exp2_approx(v.y));  // exp(-a^2 / 2)
    const float2 q = __fmul2_rn(r, e);                                 // Phi(-a)
    const float2 c = __ffma2_rn(q, both(-1.0f), both(1.0f));
    const float2 p = make_float2(x.x < 0.0f ? q.x : c.x, x.y < 0.0f ? q.y : c.y);
    f = __fmul2_rn(x, p);
    if (DERIV) d = __ffma2_rn(__fmul2_rn(x, both(0.39894228f)), e, p);
  } else {
    constexpr bool kScaled = DT != GC_F16;
    const float2 v = kScaled ? __ffma2_rn(x, both(-1.44269504f), both(-8.0f))
                             : __fmul2_rn(x, both(-1.44269504f));
    const float2 u = __fadd2_rn(make_float2(exp2_approx(v.x), exp2_approx(v.y)),
                                both(kScaled ? 0.00390625f : 1.0f));
    float2 s = make_float2(rcp_approx(u.x), rcp_approx(u.y));
    if (kScaled) s = __fmul2_rn(s, both(0.00390625f));
    f = __fmul2_rn(x, s);
    if (DERIV) d = __ffma2_rn(f, __ffma2_rn(s, both(-1.0f), both(1.0f)), s);
  }
}

// One tensor [rows, cols]: base address and row stride in bytes, its end.
struct Mat {
  char* p;
  int64_t pitch;
  const char* end;
};

struct Args {
  Mat x, gate, y;  // forward: inputs, output; backward: dy in x, dgate in gate, dx in y
  uint8_t *codes, *scales, *gate_codes, *gate_scales;
  int64_t row_bytes, codes_pitch, scales_pitch;
  uint32_t total;  // runs of all rows
  uint32_t runs;   // of one row
};

// The warp's run: its row, first byte in the row, whether it lies inside.
template <int U, bool ALIGNED>
struct Run {
  int64_t row;
  uint32_t at;
  bool any, inner;
  __device__ __forceinline__ Run(const Args& a) {
    const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const uint32_t id = blockIdx.x * (kThreads / 32) + warp;
    any = id < a.total;
    row = id / a.runs;
    const uint32_t run = id - (uint32_t)row * a.runs;
    at = run * (U * 512u);
    inner = (int64_t)at + U * 512 + (ALIGNED ? 0 : 16) <= a.row_bytes;
  }
};

// Bytes of codes of a run before unit i * 32 + lane.
template <int DT>
__device__ __forceinline__ uint32_t code_at(int i) {
  return (uint32_t)(i * 32 + (threadIdx.x & 31)) * Elem<DT>::V;
}

template <int DT, int U, bool ALIGNED>
__device__ __forceinline__ void save_run(const uint4 (&r)[U], uint8_t* codes, uint8_t* scales,
                                         const Args& a, const Run<U, ALIGNED>& run) {
  constexpr int V = Elem<DT>::V;
  const int64_t c0 = run.at / elem_size(DT);
  uint8_t* pc = codes + run.row * a.codes_pitch + c0;
  uint8_t* ps = scales + run.row * a.scales_pitch + c0 / kActGroup;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float v[V];
    Elem<DT>::unpack(r[i], v);
    const uint32_t b = scale_byte(group_max_bits<DT>(r[i])), c = code_at<DT>(i);
    if (run.inner || c0 + c < a.codes_pitch) {
      store_codes<DT>(pc + c, r[i], v, b);
      if ((c & (kActGroup - 1)) == 0) ps[c / kActGroup] = (uint8_t)b;
    }
  }
}

// Blocks per SM: 64 registers hold two tensors' units, 48 one's, 40 those of a
// save alone.  (Left to the compiler, GELU's gated form took 70: 8192 x 11008
// bf16 131 us instead of 121; with 42, a save of 8192 x 4096 fp32 36 instead
// of 34.)
constexpr int forward_blocks(int kind, bool gated) { return kind == kKindNone ? 6 : gated ? 4 : 5; }

template <int DT, int KIND, bool GATED, bool ALIGNED, int U>
__global__ void __launch_bounds__(kThreads, forward_blocks(KIND, GATED))
    act_forward_kernel(const __grid_constant__ Args a) {
  constexpr int V = Elem<DT>::V;
  const Run<U, ALIGNED> run(a);
  if (!run.any) return;
  uint4 x[U], g[U];
  load_run<DT, ALIGNED>(x, a.x.p + run.row * a.x.pitch, run.at, run.inner, a.row_bytes, a.x.end);
  if (GATED)
    load_run<DT, ALIGNED>(g, a.gate.p + run.row * a.gate.pitch, run.at, run.inner, a.row_bytes,
                          a.gate.end);
  if (a.codes) {
    save_run<DT>(x, a.codes, a.scales, a, run);
    if (GATED) save_run<DT>(g, a.gate_codes, a.gate_scales, a, run);
  }
  if constexpr (KIND != kKindNone) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float2 v[V / 2], w[V / 2], d;
      unpack2<DT>(x[i], v);
      if (GATED) unpack2<DT>(g[i], w);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        float2 f;
        act<DT, KIND, false>(v[j], f, d);
        v[j] = GATED ? __fmul2_rn(f, w[j]) : f;
      }
      x[i] = pack2<DT>(v);
    }
    store_run<DT, ALIGNED>(a.y.p + run.row * a.y.pitch, run.at, run.inner, a.row_bytes, x);
  }
}

template <int V, int U>
struct Saved {
  Codes<V> c[U];
  uint32_t b[U];
};
template <int DT, int U, bool ALIGNED>
__device__ __forceinline__ void saved_run(Saved<Elem<DT>::V, U>& s, const uint8_t* codes,
                                          const uint8_t* scales, const Args& a,
                                          const Run<U, ALIGNED>& run) {
  const int64_t c0 = run.at / elem_size(DT);
  const uint8_t* pc = codes + run.row * a.codes_pitch + c0;
  const uint8_t* ps = scales + run.row * a.scales_pitch + c0 / kActGroup;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t c = code_at<DT>(i);
    s.c[i] = Codes<Elem<DT>::V>{};
    s.b[i] = 0u;
    if (run.inner || c0 + c < a.codes_pitch) {
      s.c[i] = load_codes<Elem<DT>::V>(pc + c);
      s.b[i] = __ldg(ps + c / kActGroup);
    }
  }
}

// KIND == kKindNone: restore.
template <int DT, int KIND, bool GATED, bool ALIGNED, int U>
__global__ void __launch_bounds__(kThreads, 5)
    act_backward_kernel(const __grid_constant__ Args a) {
  constexpr int V = Elem<DT>::V;
  const Run<U, ALIGNED> run(a);
  if (!run.any) return;
  uint4 r[U], h[U];
  Saved<V, U> sx, sg;
  if (KIND != kKindNone)
    load_run<DT, ALIGNED>(r, a.x.p + run.row * a.x.pitch, run.at, run.inner, a.row_bytes,
                          a.x.end);
  saved_run<DT>(sx, a.codes, a.scales, a, run);
  if (GATED) saved_run<DT>(sg, a.gate_codes, a.gate_scales, a, run);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float2 x[V / 2];
    decode<V>(x, sx.c[i], sx.b[i]);
    if (KIND != kKindNone) {
      float2 dy[V / 2], g[V / 2], dg[V / 2];
      unpack2<DT>(r[i], dy);
      if (GATED) decode<V>(g, sg.c[i], sg.b[i]);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        float2 f, d;
        act<DT, KIND, true>(x[j], f, d);
        if (GATED) dg[j] = __fmul2_rn(dy[j], f);
        x[j] = __fmul2_rn(GATED ? __fmul2_rn(dy[j], g[j]) : dy[j], d);
      }
      if (GATED) h[i] = pack2<DT>(dg);
    }
    r[i] = pack2<DT>(x);
  }
  store_run<DT, ALIGNED>(a.y.p + run.row * a.y.pitch, run.at, run.inner, a.row_bytes, r);
  if (GATED)
    store_run<DT, ALIGNED>(a.gate.p + run.row * a.gate.pitch, run.at, run.inner, a.row_bytes, h);
}

// --- host ----------------------------------------------------------------------------------------

// Units per lane of a long run.  The gated backward kernel of the 16-bit types
// holds five tensors' units in 48 registers, and takes three: with four it
// keeps 140 bytes of them in local memory (8192 x 11008 bf16 SiLU 137 us
// instead of 131, 8192 x 4096 56 instead of 54).
constexpr int unroll(int dtype, bool gated, bool back) {
  return back && gated && dtype != GC_F32 ? 3 : 4;
}

template <int DT, int KIND, bool GATED, bool BACK, bool ALIGNED>
gc_status launch_sized(gc_ctx* ctx, Args a, int64_t rows) {
  const int64_t segs = ceil_div(a.codes_pitch / Elem<DT>::V, 32);  // of 32 units, per row
  // long runs where a row has one and every SM gets at least two blocks of
  // them; else a unit per lane (17 x 4096 bf16: 34 blocks instead of 9)
  constexpr int kUnroll = unroll(DT, GATED, BACK);
  const int64_t runs = ceil_div(segs, kUnroll);
  const bool large = segs >= kUnroll && rows * runs >= (int64_t)ctx->num_sms * 16;
  a.runs = (uint32_t)(large ? runs : segs);
  // (a matrix of as many runs would take 2 TB)
  if (rows * a.runs > UINT32_MAX - kThreads / 32) return GC_ERR_UNSUPPORTED;
  a.total = (uint32_t)(rows * a.runs);
  const unsigned g = (unsigned)ceil_div(rows * a.runs, (int64_t)(kThreads / 32));
  if (BACK) {
    if (large)
      act_backward_kernel<DT, KIND, GATED, ALIGNED, kUnroll><<<g, kThreads, 0, ctx->stream>>>(a);
    else
      act_backward_kernel<DT, KIND, GATED, ALIGNED, 1><<<g, kThreads, 0, ctx->stream>>>(a);
  } else {
    if (large)
      act_forward_kernel<DT, KIND, GATED, ALIGNED, kUnroll><<<g, kThreads, 0, ctx->stream>>>(a);
    else
      act_forward_kernel<DT, KIND, GATED, ALIGNED, 1><<<g, kThreads, 0, ctx->stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

template <int KIND, bool GATED, bool BACK>
gc_status launch_typed(gc_ctx* ctx, const Args& a, int64_t rows, int dtype, bool aligned) {
  if (dtype == GC_F32)
    return aligned ? launch_sized<GC_F32, KIND, GATED, BACK, true>(ctx, a, rows)
                   : launch_sized<GC_F32, KIND, GATED, BACK, false>(ctx, a, rows);
  if (dtype == GC_BF16)
    return aligned ? launch_sized<GC_BF16, KIND, GATED, BACK, true>(ctx, a, rows)
                   : launch_sized<GC_BF16, KIND, GATED, BACK, false>(ctx, a, rows);
  return aligned ? launch_sized<GC_F16, KIND, GATED, BACK, true>(ctx, a, rows)
                 : launch_sized<GC_F16, KIND, GATED, BACK, false>(ctx, a, rows);
}

Mat mat(const void* p, int64_t ld, int dtype, int64_t rows, int64_t cols) {
  const int e = elem_size(dtype);
  char* c = static_cast<char*>(const_cast<void*>(p));
  return {c, ld * e, c + ((rows - 1) * ld + cols) * e};
}

Args common(int dtype, int64_t cols) {
  Args a{};
  a.row_bytes = cols * elem_size(dtype);
  a.codes_pitch = ckpt_codes_pitch(cols);
  a.scales_pitch = ckpt_scales_pitch(cols);
  return a;
}

}  // namespace

gc_status launch_ckpt_save(gc_ctx* ctx, const void* x, int dtype, int64_t rows, int64_t cols,
                           int64_t ldx, uint8_t* codes, uint8_t* scales) {
  if (rows == 0 || cols == 0) return GC_OK;
  Args a = common(dtype, cols);
  a.x = mat(x, ldx, dtype, rows, cols);
  a.codes = codes;
  a.scales = scales;
  LaunchScope L(ctx, GC_PHASE_CKPT_SAVE);
  return launch_typed<kKindNone, false, false>(ctx, a, rows, dtype, row_aligned(ldx, dtype));
}

gc_status launch_ckpt_restore(gc_ctx* ctx, const uint8_t* codes, const uint8_t* scales, int dtype,
                              int64_t rows, int64_t cols, void* x_out, int64_t ldx) {
  if (rows == 0 || cols == 0) return GC_OK;
  Args a = common(dtype, cols);
  a.y = mat(x_out, ldx, dtype, rows, cols);
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  LaunchScope L(ctx, GC_PHASE_CKPT_RESTORE);
  return launch_typed<kKindNone, false, true>(ctx, a, rows, dtype, row_aligned(ldx, dtype));
}

gc_status launch_act_forward(gc_ctx* ctx, int kind, const void* x, int64_t ldx, const void* gate,
                             int64_t ldgate, int dtype, int64_t rows, int64_t cols, void* y,
                             int64_t ldy, uint8_t* codes, uint8_t* scales, uint8_t* gate_codes,
                             uint8_t* gate_scales) {
  if (rows == 0 || cols == 0) return GC_OK;
  Args a = common(dtype, cols);
  a.x = mat(x, ldx, dtype, rows, cols);
  if (gate) a.gate = mat(gate, ldgate, dtype, rows, cols);
  a.y = mat(y, ldy, dtype, rows, cols);
  a.codes = codes;
  a.scales = scales;
  a.gate_codes = gate_codes;
  a.gate_scales = gate_scales;
  const bool aligned = row_aligned(ldx, dtype) && row_aligned(ldy, dtype) &&
                       (!gate || row_aligned(ldgate, dtype));
  LaunchScope L(ctx, GC_PHASE_ACT_FORWARD);
  if (kind == GC_GELU)
    return gate ? launch_typed<GC_GELU, true, false>(ctx, a, rows, dtype, aligned)
                : launch_typed<GC_GELU, false, false>(ctx, a, rows, dtype, aligned);
  return gate ? launch_typed<GC_SILU, true, false>(ctx, a, rows, dtype, aligned)
              : launch_typed<GC_SILU, false, false>(ctx, a, rows, dtype, aligned);
}

gc_status launch_act_backward(gc_ctx* ctx, int kind, const void* dy, int64_t lddy,
                              const uint8_t* codes, const uint8_t* scales,
                              const uint8_t* gate_codes, const uint8_t* gate_scales, int dtype,
                              int64_t rows, int64_t cols, void* dx, int64_t lddx, void* dgate,
                              int64_t lddgate) {
  if (rows == 0 || cols == 0) return GC_OK;
  Args a = common(dtype, cols);
  a.x = mat(dy, lddy, dtype, rows, cols);
  if (dgate) a.gate = mat(dgate, lddgate, dtype, rows, cols);
  a.y = mat(dx, lddx, dtype, rows, cols);
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  a.gate_codes = const_cast<uint8_t*>(gate_codes);
  a.gate_scales = const_cast<uint8_t*>(gate_scales);
  const bool aligned = row_aligned(lddy, dtype) && row_aligned(lddx, dtype) &&
                       (!dgate || row_aligned(lddgate, dtype));
  LaunchScope L(ctx, GC_PHASE_ACT_BACKWARD);
  if (kind == GC_GELU)
    return dgate ? launch_typed<GC_GELU, true, true>(ctx, a, rows, dtype, aligned)
                 : launch_typed<GC_GELU, false, true>(ctx, a, rows, dtype, aligned);
  return dgate ? launch_typed<GC_SILU, true, true>(ctx, a, rows, dtype, aligned)
               : launch_typed<GC_SILU, false, true>(ctx, a, rows, dtype, aligned);
}

}  // namespace gc
