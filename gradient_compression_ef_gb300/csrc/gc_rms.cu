// gc_rms.cu -- root-mean-square norm behind the residual's addition.
//
//   forward   h = x + res (rounded to its type; h = x without res),
//             rstd = 1 / sqrt(sum(h^2) / n + eps),  y = h rstd gamma;
//             h and y are stored, saved in 8 bits (y's checkpoint is what the
//             weight gradient of the layer behind the norm reads), or both
//   backward  n_j = h_j rstd,  d_j = dy_j gamma_j,
//             dx_j = rstd (d_j - n_j sum(d n) / cols) + dres_j,
//             dgamma_j = sum over rows of dy_j n_j
//
// Each input is read once; sums are fp32, in an order that sizes alone decide.
// Bound by memory: forward 2 inputs and up to 2 outputs with their codes,
// backward 3 inputs and one output, 40 and 25 instructions per element (fp32 rows
// off 16-byte boundaries 78 and 51).
//   more rows than SMs, 2 KB  a block walks over rows that bulk copies bring
//   to 11776 (forward 15872)  into a ring of stages, a producer warp ahead of
//   columns, two rows fit     it; 16 columns per thread, gamma and the column
//                             sums in registers; backward the second pass reads
//                             the stage again
//   narrower, or few rows     a row in the registers of a warp or a block, the
//                             next one loaded ahead
//   wider still               the row is read again from L2
//
// Measured (plain copy: 6.79 TB/s), forward and backward: 16384 x 4096 bf16 with
// checkpoints 110 us (6.1 TB/s) and 76 + 5 (6.2); 3001 x 4099 fp32 on 4-byte
// boundaries 50 (4.1) and 44 + 5 (4.5), the shifting of each unit into place;
// 2048 x 11008 fp16 44 (4.1) and 40 + 6 (4.0), one block per SM, whose sum over
// 22 warps nothing hides.  Without the ring, bf16 with checkpoints: 4096 x 16384
// 166 (4.1) and 163 (2.9), 4096 x 12288 backward 146 (2.4), 64 x 4096 forward 8.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "gc_rows.cuh"

namespace gc {
namespace {

struct RmsArgs {
  const char *x, *res, *dy, *dres;  // x: the input (forward), or h (backward)
  const char *xend, *resend, *dyend, *dresend;
  char *h, *y;  // forward: outputs or NULL; backward: y is dx
  const void* gamma;
  float* rstd;
  uint8_t *codes, *scales, *ycodes, *yscales;
  float *dgamma, *part;  // [parts][part_pitch]
  int64_t rows, cols, row_bytes, xpitch, respitch, dypitch, drespitch, hpitch, ypitch;
  int64_t codes_pitch, scales_pitch, part_pitch;
  float eps;
  int ptype, accumulate;
  // ring of stages (set at launch)
  uint32_t* status;
  uint32_t second_at, third_at, scales_at, stage_bytes;  // places within a stage
  int stages;
};

// A unit's part of a checkpoint, column c on; every lane of the warp calls it.
template <int DT>
__device__ __forceinline__ void save_unit(uint8_t* codes, uint8_t* scales, const uint4& r,
                                          int64_t c, int64_t pitch) {
  constexpr int V = Elem<DT>::V;
  const uint32_t sb = scale_byte(group_max_bits<DT>(r));
  if (c >= pitch) return;
  float v[V];
  Elem<DT>::unpack(r, v);
  store_codes<DT>(codes + c, r, v, sb);
  if ((threadIdx.x & 31) % (kActGroup / V) == 0) scales[c / kActGroup] = (uint8_t)sb;
}

template <int DT>
__device__ __forceinline__ uint4 add_units(const uint4& a, const uint4& b) {
  constexpr int H = Elem<DT>::V / 2;
  float2 u[H], v[H];
  unpack2<DT>(a, u);
  unpack2<DT>(b, v);
#pragma unroll
  for (int j = 0; j < H; ++j) u[j] = __fadd2_rn(u[j], v[j]);
  return pack2<DT>(u);
}

template <int DT>
__device__ __forceinline__ float2 add_squares(const uint4& r, float2 s) {
  constexpr int H = Elem<DT>::V / 2;
  float2 v[H];
  unpack2<DT>(r, v);
#pragma unroll
  for (int j = 0; j < H; ++j) s = __ffma2_rn(v[j], v[j], s);
  return s;
}

// 1 / sqrt(sum / n + eps) as two terms, the second one what the first lacks:
// y may lie next to a border of its rounding, or of its code.
struct Rstd {
  float hi, lo;
};
struct Count {  // 1 / n as two terms
  float hi, lo;
  __device__ __forceinline__ explicit Count(int64_t n)
      : hi(1.0f / (float)n), lo(fmaf(-hi, (float)n, 1.0f) * hi) {}
};
__device__ __forceinline__ Rstd rstd_of(float sum, const Count& n, float eps) {
  const float v = fmaf(sum, n.hi, (sum <= FLT_MAX ? sum * n.lo : 0.0f) + eps);
  const float r = rsqrtf(v);
  const float q = __fmul_rn(r, r);
  const float e = fmaf(-v, fmaf(r, r, -q), fmaf(-v, q, 1.0f));  // 1 - v r^2
  return {r, fabsf(e) < 1.0f ? 0.5f * r * e : 0.0f};  // not where r is 0 or infinite
}

// y's unit from h's: h rstd as two terms, times gamma, rounded once to fp32.
// CLAMP: the small term is kept finite: where gamma or rstd is infinite it would
// be a NaN, or an infinity of the other sign, beside the large one.
template <int DT, bool CLAMP>
__device__ __forceinline__ uint4 scaled(const uint4& r, const Rstd& rstd,
                                        const float (&g)[Elem<DT>::V]) {
  constexpr int H = Elem<DT>::V / 2;
  float2 v[H];
  unpack2<DT>(r, v);
#pragma unroll
  for (int j = 0; j < H; ++j) {
    const float2 w = make_float2(g[2 * j], g[2 * j + 1]);
    const float2 p = __fmul2_rn(v[j], both(rstd.hi));
    const float2 minus = make_float2(-p.x, -p.y);
    float2 q = __ffma2_rn(v[j], both(rstd.lo), __ffma2_rn(v[j], both(rstd.hi), minus));
    q = __fmul2_rn(q, w);
    if (CLAMP)
      q = make_float2(fminf(fmaxf(q.x, -FLT_MAX), FLT_MAX), fminf(fmaxf(q.y, -FLT_MAX), FLT_MAX));
    v[j] = __ffma2_rn(p, w, q);
  }
  return pack2<DT>(v);
}
// Whether a thread's parameters are all finite.
template <int V>
__device__ __forceinline__ bool all_finite(const float (&g)[V]) {
  bool yes = true;
#pragma unroll
  for (int j = 0; j < V; ++j) yes = yes && fabsf(g[j]) <= FLT_MAX;
  return yes;
}
template <int K, int V>
__device__ __forceinline__ bool all_finite(const float (&g)[K][V]) {
  bool yes = true;
#pragma unroll
  for (int i = 0; i < K; ++i) yes = yes && all_finite(g[i]);
  return yes;
}
// (Clamping everywhere: 16384 x 4096 bf16, forward and backward, 229 -> 232 us.)
template <int DT>
__device__ __forceinline__ uint4 scale_unit(const uint4& r, const Rstd& rstd,
                                            const float (&g)[Elem<DT>::V], bool finite) {
  return finite && rstd.hi <= FLT_MAX ? scaled<DT, false>(r, rstd, g) : scaled<DT, true>(r, rstd, g);
}

// A row per team: a warp (U units per lane), or a block.
template <int DT, bool WARP, int U, bool ALIGNED>
__global__ void __launch_bounds__(WARP ? 256 : 1024)
    rms_forward_kernel(const __grid_constant__ RmsArgs a) {
  constexpr int V = Elem<DT>::V;
  __shared__ float2 slot[2][32];
  RowSum<WARP> sum{slot};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t at = WARP ? 0u : (uint32_t)warp * (512u * U);
  const bool inner = (int64_t)at + 512 * U + (ALIGNED ? 0 : 16) <= a.row_bytes;
  const int64_t c0 = at / elem_size(DT) + lane * V;
  const int64_t step = WARP ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
  const Count n(a.cols);
  uint4 u[U], v[U];
  auto load = [&](int64_t r) {
    load_run<DT, ALIGNED>(u, a.x + r * a.xpitch, at, inner, a.row_bytes, a.xend);
    if (a.res) load_run<DT, ALIGNED>(v, a.res + r * a.respitch, at, inner, a.row_bytes, a.resend);
  };
  if (row < a.rows) load(row);
  float g[U][V];
#pragma unroll
  for (int i = 0; i < U; ++i)
    load_params<V>(g[i], a.gamma, a.ptype, c0 + i * 32 * V, a.cols, 1.0f);
  const bool finite = all_finite(g);
  for (; row < a.rows; row += step) {
    uint4 h[U];
#pragma unroll
    for (int i = 0; i < U; ++i) h[i] = a.res ? add_units<DT>(u[i], v[i]) : u[i];
    if (row + step < a.rows) load(row + step);
    float2 s = both(0.0f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      s = add_squares<DT>(h[i], s);
      keep_packed(h[i]);
    }
    const Rstd rstd = rstd_of(sum(s.x + s.y), n, a.eps);
    if (WARP ? lane == 0 : threadIdx.x == 0) a.rstd[row] = rstd.hi + rstd.lo;
    if (a.h) store_run<DT, ALIGNED>(a.h + row * a.hpitch, at, inner, a.row_bytes, h);
    if (a.codes) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        save_unit<DT>(a.codes + row * a.codes_pitch, a.scales + row * a.scales_pitch, h[i],
                      c0 + i * 32 * V, a.codes_pitch);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) h[i] = scale_unit<DT>(h[i], rstd, g[i], finite);
    if (a.y) store_run<DT, ALIGNED>(a.y + row * a.ypitch, at, inner, a.row_bytes, h);
    if (a.ycodes) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        save_unit<DT>(a.ycodes + row * a.codes_pitch, a.yscales + row * a.scales_pitch, h[i],
                      c0 + i * 32 * V, a.codes_pitch);
    }
  }
}

// Rows wider than a block's registers: the inputs are read again (from L2) for
// the second pass.
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(1024)
    rms_forward_wide_kernel(const __grid_constant__ RmsArgs a) {
  constexpr int V = Elem<DT>::V;
  __shared__ float2 slot[2][32];
  RowSum<false> sum{slot};
  const int64_t round = (int64_t)blockDim.x * 16;
  const Count n(a.cols);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char *x = a.x + row * a.xpitch, *res = a.res + (a.res ? row * a.respitch : 0);
    auto get = [&](int64_t off) {
      uint4 r = load_unit<DT, ALIGNED>(x, off, a.row_bytes, a.xend);
      if (a.res) r = add_units<DT>(r, load_unit<DT, ALIGNED>(res, off, a.row_bytes, a.resend));
      return r;
    };
    float2 s = both(0.0f);
    for (int64_t b = 0; b < a.row_bytes; b += round)
      s = add_squares<DT>(get(b + threadIdx.x * 16), s);
    const Rstd rstd = rstd_of(sum(s.x + s.y), n, a.eps);
    if (threadIdx.x == 0) a.rstd[row] = rstd.hi + rstd.lo;
    for (int64_t b = 0; b < a.row_bytes; b += round) {
      const int64_t off = b + threadIdx.x * 16, c = off / elem_size(DT);
      const uint4 h = get(off);
      if (a.h) store_unit<DT, ALIGNED>(a.h + row * a.hpitch, off, a.row_bytes, h);
      if (a.codes)
        save_unit<DT>(a.codes + row * a.codes_pitch, a.scales + row * a.scales_pitch, h, c,
                      a.codes_pitch);
      float g[V];
      load_params<V>(g, a.gamma, a.ptype, c, a.cols, 1.0f);
      const uint4 y = scale_unit<DT>(h, rstd, g, all_finite(g));
      if (a.y) store_unit<DT, ALIGNED>(a.y + row * a.ypitch, off, a.row_bytes, y);
      if (a.ycodes)
        save_unit<DT>(a.ycodes + row * a.codes_pitch, a.yscales + row * a.scales_pitch, y, c,
                      a.codes_pitch);
    }
  }
}

// --- rows through a ring of stages ---------------------------------------------------------------

constexpr int kMaxStages = 6;
constexpr int kCols = 16;          // columns per thread
// Registers a thread: the first where a block's warps fit with them, the second
// for wider rows.  (A kernel that spills pays twice beside a ring: shared memory
// leaves the L1 nothing to keep the spilled in.  Backward at 72 registers, three
// blocks per SM, 3001 x 4099 fp32: 59 us, at 96, two blocks: 45.)
constexpr int kForwardRegs[2] = {80, 64}, kBackwardRegs[2] = {96, 80};
// warps that an SM's four register files hold
constexpr int warps_at(int regs) { return 16384 / (32 * regs) * 4; }

// One thread's part: row `row` into a stage.  Forward: x, res.  BACK: dy,
// dres, then h or its checkpoint.
template <int DT, bool BACK, bool CKPT>
__device__ __forceinline__ void fill_stage(const RmsArgs& a, int64_t row, char* stage,
                                           uint64_t* full) {
  using namespace sm100;
  const char* r0 = BACK ? a.dy + row * a.dypitch : a.x + row * a.xpitch;
  const char* r1 = BACK ? a.dres + row * a.drespitch : a.res + row * a.respitch;
  const char* r2 = a.x + row * a.xpitch;
  const bool second = BACK ? a.dres != nullptr : a.res != nullptr;
  const uint32_t n0 = bulk_size<DT>(r0, a.row_bytes, BACK ? a.dyend : a.xend, stage);
  uint32_t n1 = 0, n2 = 0, n3 = 0;
  if (second)
    n1 = bulk_size<DT>(r1, a.row_bytes, BACK ? a.dresend : a.resend, stage + a.second_at);
  if (BACK && CKPT) {
    n2 = (uint32_t)a.codes_pitch;
    n3 = (uint32_t)a.scales_pitch;
  } else if (BACK) {
    n2 = bulk_size<DT>(r2, a.row_bytes, a.xend, stage + a.third_at);
  }
  mbar_arrive_expect_tx(full, n0 + n1 + n2 + n3);
  auto from = [](const char* r) { return r - (reinterpret_cast<uintptr_t>(r) & 15u); };
  if (n0) bulk_load(stage, from(r0), n0, full);
  if (n1) bulk_load(stage + a.second_at, from(r1), n1, full);
  if (BACK && CKPT) {
    bulk_load(stage + a.third_at, a.codes + row * a.codes_pitch, n2, full);
    bulk_load(stage + a.scales_at, a.scales + row * a.scales_pitch, n3, full);
  } else if (n2) {
    bulk_load(stage + a.third_at, from(r2), n2, full);
  }
}

// The producer warp: copies the block's rows, stage after stage, as the row's
// warps hand the stages back.
template <int DT, bool BACK, bool CKPT>
__device__ __forceinline__ bool produce(const RmsArgs& a, char* stages, uint64_t* full,
                                        uint64_t* empty) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) {
    RingPos ring;
    int filled = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ring.next(a.stages)) {
      if (filled < a.stages) {
        ++filled;
      } else {
        if (!sm100::mbar_wait(&empty[ring.st], ring.ph ^ 1u, kWaitCycles)) {
          ok = false;
          break;
        }
        // the warps read the stage through the generic proxy, the copy
        // refills it through the asynchronous one
        sm100::fence_proxy_async_smem();
      }
      fill_stage<DT, BACK, CKPT>(a, row, stages + ring.st * a.stage_bytes, &full[ring.st]);
    }
  }
  return ok;
}

// The ring's barriers and the sums' slots; the whole block calls it.
__device__ __forceinline__ void ring_begin(const RmsArgs& a, float (&slot)[2][36], uint64_t* full,
                                           uint64_t* empty) {
  for (int i = threadIdx.x; i < 72; i += blockDim.x) slot[i / 36][i % 36] = 0.0f;
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      sm100::mbar_init(&full[i], 1);
      sm100::mbar_init(&empty[i], (blockDim.x - 32) / 32);
    }
    sm100::mbar_fence_init();
  }
  __syncthreads();
}

// Where in its 16 bytes a row begins.
__device__ __forceinline__ uint32_t shift_of(const char* p, int64_t pitch, int64_t row) {
  return ((uint32_t)reinterpret_cast<uintptr_t>(p) + (uint32_t)row * (uint32_t)pitch) & 15u;
}

template <int DT, int ROWS, int REGS>
__global__ void __maxnreg__(REGS)
    rms_forward_ring_kernel(const __grid_constant__ RmsArgs a) {
  using namespace sm100;
  constexpr int V = Elem<DT>::V, K = kCols / V;
  extern __shared__ __align__(128) char stages[];
  __shared__ __align__(16) float slot[2][36];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  const int t = threadIdx.x, nt = blockDim.x - 32;  // the last warp is the producer
  ring_begin(a, slot, full, empty);
  if (t >= nt) {
    ring_end(produce<DT, false, false>(a, stages, full, empty), a.status);
    return;
  }
  RowsSum<1> sum{slot, nt};
  const uint32_t u0 = (t & ~31) * K, u1 = u0 + (t & 31);  // the warp's and the thread's first unit
  const uint32_t base = smem_u32(stages) + u1 * 16;
  const Count n(a.cols);
  float g[K][V];
  // bytes of the row from the first unit on
  const int rest = (int)min((int64_t)(1 << 30), a.row_bytes - (int64_t)u1 * 16);
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int64_t u = u1 + i * 32;
    load_params<V>(g[i], a.gamma, a.ptype, u * V, a.cols, 1.0f);
  }
  const bool finite = all_finite(g);
  bool ok = true;
  RingPos ring;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    ok = mbar_wait(&full[ring.st], ring.ph, kWaitCycles);
    const uint32_t stage = base + ring.st * a.stage_bytes;
    const uint32_t mis0 = ROWS == kAnywhere ? shift_of(a.x, a.xpitch, row) : 0u;
    const uint32_t mis1 = ROWS == kAnywhere ? shift_of(a.res, a.respitch, row) : 0u;
    uint4 h[K];
    float2 q = both(0.0f);
#pragma unroll
    for (int i = 0; i < K; ++i) {
      h[i] = make_uint4(0u, 0u, 0u, 0u);
      if (ROWS == kFull || rest - i * 512 > 0) {
        h[i] = staged_unit<DT, ROWS>(stage + i * 512, mis0, rest - i * 512);
        if (a.res)
          h[i] = add_units<DT>(
              h[i], staged_unit<DT, ROWS>(stage + a.second_at + i * 512, mis1, rest - i * 512));
      }
      q = add_squares<DT>(h[i], q);
      keep_packed(h[i]);
    }
    // the warp holds its part of the row
    __syncwarp();
    if ((t & 31) == 0) mbar_arrive(&empty[ring.st]);
    ring.next(a.stages);
    if (a.h) put_units<DT, ROWS>(a.h + row * a.hpitch, u0, a.row_bytes, h);
    if (a.codes) {
#pragma unroll
      for (int i = 0; i < K; ++i)
        save_unit<DT>(a.codes + row * a.codes_pitch, a.scales + row * a.scales_pitch, h[i],
                      (int64_t)(u1 + i * 32) * V, a.codes_pitch);
    }
    float s[1] = {q.x + q.y};
    sum(s, ok);
    if (!ok) break;
    const Rstd rstd = rstd_of(s[0], n, a.eps);
    if (t == 0) a.rstd[row] = rstd.hi + rstd.lo;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      keep_packed(h[i]);
      h[i] = scale_unit<DT>(h[i], rstd, g[i], finite);
    }
    if (a.y) put_units<DT, ROWS>(a.y + row * a.ypitch, u0, a.row_bytes, h);
    if (a.ycodes) {
#pragma unroll
      for (int i = 0; i < K; ++i)
        save_unit<DT>(a.ycodes + row * a.codes_pitch, a.yscales + row * a.scales_pitch, h[i],
                      (int64_t)(u1 + i * 32) * V, a.codes_pitch);
    }
  }
  ring_end(ok, a.status);
}

// --- backward ------------------------------------------------------------------------------------

// A unit of h as it lies in memory, whole or in 8 bits.
template <int DT, bool CKPT>
struct Kept {
  uint4 raw;
  __device__ __forceinline__ void values(float2 (&v)[Elem<DT>::V / 2]) const {
    unpack2<DT>(raw, v);
  }
};
template <int DT>
struct Kept<DT, true> {
  Codes<Elem<DT>::V> c;
  uint32_t b;
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int64_t col,
                                       int64_t pitch) {
#pragma unroll
    for (int i = 0; i < Elem<DT>::V / 4; ++i) c.w[i] = 0u;
    b = 0u;
    if (col >= pitch) return;
    c = load_codes<Elem<DT>::V>(codes + col);
    b = __ldg(scales + col / kActGroup);
  }
  __device__ __forceinline__ void values(float2 (&v)[Elem<DT>::V / 2]) const {
    decode<Elem<DT>::V>(v, c, b);
  }
};

template <int DT, bool CKPT, bool ALIGNED, int U>
__device__ __forceinline__ void load_kept(Kept<DT, CKPT> (&k)[U], const RmsArgs& a, int64_t row,
                                          uint32_t at, bool inner, int64_t c0) {
  constexpr int V = Elem<DT>::V;
  if constexpr (CKPT) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      k[i].load(a.codes + row * a.codes_pitch, a.scales + row * a.scales_pitch, c0 + i * 32 * V,
                a.codes_pitch);
  } else {
    uint4 r[U];
    load_run<DT, ALIGNED>(r, a.x + row * a.xpitch, at, inner, a.row_bytes, a.xend);
#pragma unroll
    for (int i = 0; i < U; ++i) k[i].raw = r[i];
  }
}

// Columns past the row's end have dy = 0 and must not spoil the sums, whatever
// a checkpoint's last group holds (a NaN group restores as NaN throughout).
template <int DT>
__device__ __forceinline__ void mask_values(float2 (&v)[Elem<DT>::V / 2], int64_t left) {
  if (left >= Elem<DT>::V) return;
#pragma unroll
  for (int j = 0; j < Elem<DT>::V / 2; ++j) {
    if (2 * j >= left) v[j].x = 0.0f;
    if (2 * j + 1 >= left) v[j].y = 0.0f;
  }
}

// A block's column sums: to its partial row, or, where it is the only block,
// to the gradient.
__device__ __forceinline__ void put_sum(const RmsArgs& a, int64_t c, float g) {
  if (c >= a.cols) return;
  if (gridDim.x > 1) a.part[blockIdx.x * a.part_pitch + c] = g;
  else a.dgamma[c] = a.accumulate ? a.dgamma[c] + g : g;
}

template <int DT, bool CKPT, bool WARP, int U, bool ALIGNED>
__global__ void __launch_bounds__(WARP ? 256 : 512)
    rms_backward_kernel(const __grid_constant__ RmsArgs a) {
  constexpr int V = Elem<DT>::V, H = V / 2;
  constexpr bool kAhead = U <= 2;  // next row's loads and gamma in registers
  __shared__ float2 slot[2][32];
  extern __shared__ __align__(16) float sums[];  // WARP: [warps][U * 32 * V]
  RowSum<WARP> sum{slot};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t at = WARP ? 0u : (uint32_t)warp * (512u * U);
  const bool inner = (int64_t)at + 512 * U + (ALIGNED ? 0 : 16) <= a.row_bytes;
  const int64_t c0 = at / elem_size(DT) + lane * V;
  const int64_t step = WARP ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
  const float inv_n = 1.0f / (float)a.cols;
  uint4 ndy[U], ndres[U];
  Kept<DT, CKPT> nk[U];
  float nrstd = 0.0f;
  auto load = [&](int64_t r) {
    load_run<DT, ALIGNED>(ndy, a.dy + r * a.dypitch, at, inner, a.row_bytes, a.dyend);
    load_kept<DT, CKPT, ALIGNED>(nk, a, r, at, inner, c0);
    if (a.dres)
      load_run<DT, ALIGNED>(ndres, a.dres + r * a.drespitch, at, inner, a.row_bytes, a.dresend);
    nrstd = a.rstd[r];
  };
  if (kAhead && row < a.rows) load(row);
  float g[kAhead ? U : 1][V];
  if (kAhead) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      load_params<V>(g[kAhead ? i : 0], a.gamma, a.ptype, c0 + i * 32 * V, a.cols, 1.0f);
  }
  float2 acc[U][H];
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int j = 0; j < H; ++j) acc[i][j] = both(0.0f);
  for (; row < a.rows; row += step) {
    if (!kAhead) load(row);
    uint4 dy[U], dres[U];
    Kept<DT, CKPT> k[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      dy[i] = ndy[i];
      dres[i] = ndres[i];
      k[i] = nk[i];
    }
    const float rstd = nrstd;
    if (kAhead && row + step < a.rows) load(row + step);
    float2 s = both(0.0f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (!kAhead) load_params<V>(g[0], a.gamma, a.ptype, c0 + i * 32 * V, a.cols, 1.0f);
      const float(&gi)[V] = g[kAhead ? i : 0];
      float2 d[H], n[H];
      unpack2<DT>(dy[i], d);
      k[i].values(n);
      if (!inner) mask_values<DT>(n, a.cols - c0 - i * 32 * V);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        n[j] = __fmul2_rn(n[j], both(rstd));
        const float2 t = __fmul2_rn(d[j], n[j]);
        acc[i][j] = __fadd2_rn(acc[i][j], t);
        s = __ffma2_rn(t, make_float2(gi[2 * j], gi[2 * j + 1]), s);
      }
      keep_packed(dy[i]);
    }
    const float2 m = both(-sum(s.x + s.y) * inv_n);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (!kAhead) load_params<V>(g[0], a.gamma, a.ptype, c0 + i * 32 * V, a.cols, 1.0f);
      const float(&gi)[V] = g[kAhead ? i : 0];
      float2 d[H], n[H], r[H];
      unpack2<DT>(dy[i], d);
      k[i].values(n);
      if (a.dres) unpack2<DT>(dres[i], r);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        n[j] = __fmul2_rn(n[j], both(rstd));
        d[j] = __fmul2_rn(d[j], make_float2(gi[2 * j], gi[2 * j + 1]));
        d[j] = __ffma2_rn(n[j], m, d[j]);
        d[j] = a.dres ? __ffma2_rn(d[j], both(rstd), r[j]) : __fmul2_rn(d[j], both(rstd));
      }
      dy[i] = pack2<DT>(d);
    }
    store_run<DT, ALIGNED>(a.y + row * a.ypitch, at, inner, a.row_bytes, dy);
  }
  if (!a.dgamma) return;
  if (WARP) {
    float* mine = sums + warp * (U * 32 * V);
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int j = 0; j < H; ++j)
        *reinterpret_cast<float2*>(mine + (i * 32 + lane) * V + 2 * j) = acc[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < U * 32 * V; c += blockDim.x) {
      float t = 0.0f;
      for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += sums[w * (U * 32 * V) + c];
      put_sum(a, c, t);
    }
  } else {
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int j = 0; j < H; ++j) {
        put_sum(a, c0 + i * 32 * V + 2 * j, acc[i][j].x);
        put_sum(a, c0 + i * 32 * V + 2 * j + 1, acc[i][j].y);
      }
  }
}

// The same through the ring: dy and h are read from the stage in both passes,
// so that a thread keeps gamma and the column sums alone.
template <int DT, bool CKPT, int ROWS, int REGS>
__global__ void __maxnreg__(REGS)
    rms_backward_ring_kernel(const __grid_constant__ RmsArgs a) {
  using namespace sm100;
  constexpr int V = Elem<DT>::V, K = kCols / V, H = V / 2;
  extern __shared__ __align__(128) char stages[];
  __shared__ __align__(16) float slot[2][36];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  const int t = threadIdx.x, nt = blockDim.x - 32;  // the last warp is the producer
  ring_begin(a, slot, full, empty);
  if (t >= nt) {
    ring_end(produce<DT, true, CKPT>(a, stages, full, empty), a.status);
    return;
  }
  RowsSum<1> sum{slot, nt};
  const uint32_t u0 = (t & ~31) * K, u1 = u0 + (t & 31);  // the warp's and the thread's first unit
  const uint32_t base = smem_u32(stages);
  const float inv_n = 1.0f / (float)a.cols;
  float g[K][V];
  float2 acc[K][H];
  // bytes of the row from the first unit on
  const int rest = (int)min((int64_t)(1 << 30), a.row_bytes - (int64_t)u1 * 16);
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int64_t u = u1 + i * 32;
    load_params<V>(g[i], a.gamma, a.ptype, u * V, a.cols, 1.0f);
#pragma unroll
    for (int j = 0; j < H; ++j) acc[i][j] = both(0.0f);
  }
  float rstd = blockIdx.x < a.rows ? __ldg(a.rstd + blockIdx.x) : 0.0f;
  bool ok = true;
  RingPos ring;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float next = row + gridDim.x < a.rows ? __ldg(a.rstd + row + gridDim.x) : 0.0f;
    ok = mbar_wait(&full[ring.st], ring.ph, kWaitCycles);
    const uint32_t stage = base + ring.st * a.stage_bytes;
    const uint32_t mis0 = ROWS == kAnywhere ? shift_of(a.dy, a.dypitch, row) : 0u;
    const uint32_t mis1 = ROWS == kAnywhere ? shift_of(a.dres, a.drespitch, row) : 0u;
    const uint32_t mis2 = ROWS == kAnywhere ? shift_of(a.x, a.xpitch, row) : 0u;
    const float2 rs = both(rstd);
    // dy and n = h rstd of a unit (past the last column dy is 0)
    auto get = [&](int i, float2 (&d)[H], float2 (&n)[H]) {
      const uint32_t u = u1 + i * 32;
      unpack2<DT>(staged_unit<DT, ROWS>(stage + u * 16, mis0, rest - i * 512), d);
      if constexpr (CKPT) {
        Codes<V> c;
#pragma unroll
        for (int w = 0; w < V / 4; ++w) c.w[w] = lds_u32(stage + a.third_at + u * V + 4 * w);
        decode<V>(n, c, lds_u8(stage + a.scales_at + u / (kActGroup / V)));
      } else {
        unpack2<DT>(staged_unit<DT, ROWS>(stage + a.third_at + u * 16, mis2, rest - i * 512), n);
      }
#pragma unroll
      for (int j = 0; j < H; ++j) n[j] = __fmul2_rn(n[j], rs);
    };
    float2 q = both(0.0f);
#pragma unroll
    for (int i = 0; i < K; ++i) {
      if (ROWS != kFull && rest - i * 512 <= 0) continue;
      float2 d[H], n[H];
      get(i, d, n);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        const float2 p = __fmul2_rn(d[j], n[j]);
        acc[i][j] = __fadd2_rn(acc[i][j], p);
        q = __ffma2_rn(p, make_float2(g[i][2 * j], g[i][2 * j + 1]), q);
      }
    }
    float s[1] = {q.x + q.y};
    sum(s, ok);
    if (!ok) break;
    const float2 m = both(-s[0] * inv_n);
    uint4 res[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      res[i] = make_uint4(0u, 0u, 0u, 0u);
      if (ROWS != kFull && rest - i * 512 <= 0) continue;
      float2 d[H], n[H], r[H];
      get(i, d, n);
      if (a.dres)
        unpack2<DT>(
            staged_unit<DT, ROWS>(stage + a.second_at + (u1 + i * 32) * 16, mis1, rest - i * 512), r);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        d[j] = __fmul2_rn(d[j], make_float2(g[i][2 * j], g[i][2 * j + 1]));
        d[j] = __ffma2_rn(n[j], m, d[j]);
        d[j] = a.dres ? __ffma2_rn(d[j], rs, r[j]) : __fmul2_rn(d[j], rs);
      }
      res[i] = pack2<DT>(d);
    }
    __syncwarp();
    if ((t & 31) == 0) mbar_arrive(&empty[ring.st]);
    ring.next(a.stages);
    put_units<DT, ROWS>(a.y + row * a.ypitch, u0, a.row_bytes, res);
    rstd = next;
  }
  ring_end(ok, a.status);
  if (!a.dgamma) return;
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j)
      put_sum(a, (int64_t)(u1 + i * 32) * V + j, j & 1 ? acc[i][j / 2].y : acc[i][j / 2].x);
}

// Wider rows: two passes over the inputs, the column sums in the block's
// partial row (each place is one thread's).
template <int DT, bool CKPT, bool ALIGNED>
__global__ void __launch_bounds__(512)
    rms_backward_wide_kernel(const __grid_constant__ RmsArgs a) {
  constexpr int V = Elem<DT>::V, H = V / 2;
  __shared__ float2 slot[2][32];
  RowSum<false> sum{slot};
  const int64_t round = (int64_t)blockDim.x * 16;
  const float inv_n = 1.0f / (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char *dy = a.dy + row * a.dypitch, *dres = a.dres + (a.dres ? row * a.drespitch : 0);
    const float rstd = a.rstd[row];
    float2 d[H], n[H], r[H];
    float g[V];
    auto get = [&](int64_t off) {
      const int64_t c = off / elem_size(DT);
      Kept<DT, CKPT> k[1];
      load_kept<DT, CKPT, ALIGNED>(k, a, row, (uint32_t)off - (threadIdx.x & 31u) * 16u, false, c);
      unpack2<DT>(load_unit<DT, ALIGNED>(dy, off, a.row_bytes, a.dyend), d);
      k[0].values(n);
      mask_values<DT>(n, a.cols - c);
      load_params<V>(g, a.gamma, a.ptype, c, a.cols, 1.0f);
#pragma unroll
      for (int j = 0; j < H; ++j) n[j] = __fmul2_rn(n[j], both(rstd));
    };
    float2 s = both(0.0f);
    for (int64_t b = 0; b < a.row_bytes; b += round) {
      const int64_t off = b + threadIdx.x * 16, c = off / elem_size(DT);
      get(off);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        const float2 t = __fmul2_rn(d[j], n[j]);
        s = __ffma2_rn(t, make_float2(g[2 * j], g[2 * j + 1]), s);
        if (a.dgamma) {
          float* p = a.part + blockIdx.x * a.part_pitch + c + 2 * j;
          const bool first = row == blockIdx.x;
          if (c + 2 * j < a.cols) p[0] = first ? t.x : p[0] + t.x;
          if (c + 2 * j + 1 < a.cols) p[1] = first ? t.y : p[1] + t.y;
        }
      }
    }
    const float2 m = both(-sum(s.x + s.y) * inv_n);
    for (int64_t b = 0; b < a.row_bytes; b += round) {
      const int64_t off = b + threadIdx.x * 16;
      get(off);
      if (a.dres) unpack2<DT>(load_unit<DT, ALIGNED>(dres, off, a.row_bytes, a.dresend), r);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        d[j] = __fmul2_rn(d[j], make_float2(g[2 * j], g[2 * j + 1]));
        d[j] = __ffma2_rn(n[j], m, d[j]);
        d[j] = a.dres ? __ffma2_rn(d[j], both(rstd), r[j]) : __fmul2_rn(d[j], both(rstd));
      }
      store_unit<DT, ALIGNED>(a.y + row * a.ypitch, off, a.row_bytes, pack2<DT>(d));
    }
  }
}

// dgamma from the blocks' partial rows, in block order within each of 32
// strips, then strip by strip: 32 columns per block.
__global__ void __launch_bounds__(1024)
    rms_reduce_kernel(const __grid_constant__ RmsArgs a, int parts) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, strip = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  after_previous();
  float t = 0.0f;
  if (c < a.cols) {
#pragma unroll 4
    for (int p = strip; p < parts; p += 32) t += a.part[p * a.part_pitch + c];
  }
  s[strip][lane] = t;
  __syncthreads();
  // column `strip` of the block, a partial per lane
  t = warp_allsum(s[lane][strip]);
  const int64_t o = (int64_t)blockIdx.x * 32 + strip;
  if (lane == 0 && o < a.cols) a.dgamma[o] = a.accumulate ? a.dgamma[o] + t : t;
}

// --- host ----------------------------------------------------------------------------------------

constexpr int64_t kMaxParts = 608;  // blocks that leave a partial row, at most

struct Shape {
  bool warp, wide;
  int u;
  unsigned threads, grid;
};

// units: 16-byte units of a row; a block has up to `most` threads of up to
// `deep` units, an SM room for `per_sm` threads.
Shape pick(int64_t units, int64_t rows, int sms, int most, int deep, int per_sm) {
  Shape s{};
  if (units <= 128) {
    s.warp = true;
    s.u = units <= 32 ? 1 : units <= 64 ? 2 : 4;
    s.threads = 256;
  } else {
    s.wide = units > (int64_t)most * deep;
    s.u = units <= 2 * most ? 2 : 4;
    s.threads = s.wide ? (unsigned)most : (unsigned)round_up(ceil_div(units, (int64_t)s.u), 32);
  }
  s.grid = (unsigned)std::min<int64_t>(s.warp ? ceil_div(rows, (int64_t)8) : rows,
                                       (int64_t)sms * std::max(1, per_sm / (int)s.threads));
  return s;
}

// Rows that go through the ring: more of them than SMs (a row per block is
// loaded sooner by its own threads), not narrower than a block of 160 threads
// or so, not wider than a block's registers hold, two stages or more in shared
// memory.
struct RingPlan {
  int threads, per_sm;  // threads of the rows; 0: not this way
  int regs;             // which of the two
  unsigned smem;
};

// Dynamic shared memory that each of n blocks of an SM may use: 228 KB less
// the system's 1 KB a block and the kernels' static part.
constexpr int64_t kStaticSmem =
    (2 * 36 * sizeof(float) + 2 * kMaxStages * sizeof(uint64_t) + 127) / 128 * 128;
int64_t block_smem(int n) { return 228 * 1024 / n / 128 * 128 - 1024 - kStaticSmem; }

RingPlan plan_ring(const gc_ctx* ctx, RmsArgs& a, int dtype, bool back) {
  RingPlan p{};
  const int64_t c = ckpt_codes_pitch(a.cols);
  const int threads = (int)round_up(ceil_div(c, (int64_t)kCols), 32);
  const int* regs = back ? kBackwardRegs : kForwardRegs;
  p.regs = threads / 32 + 1 <= warps_at(regs[0]) ? 0 : 1;
  const int warps = warps_at(regs[p.regs]);
  if (a.rows <= ctx->num_sms || c * elem_size(dtype) <= 2048 || threads / 32 + 1 > warps) return p;
  const int64_t row = round_up(a.row_bytes + 30, 128);  // with a shifted start
  int64_t bytes = row;
  a.second_at = (uint32_t)bytes;
  if (back ? a.dres != nullptr : a.res != nullptr) bytes += row;
  a.third_at = (uint32_t)bytes;
  if (back) bytes += a.codes ? round_up(c, 128) : row;
  a.scales_at = (uint32_t)bytes;
  if (back && a.codes) bytes += round_up(a.scales_pitch, 128);
  a.stage_bytes = (uint32_t)bytes;
  p.per_sm = warps / (threads / 32 + 1);
  while (p.per_sm > 1 && 2 * bytes > block_smem(p.per_sm)) --p.per_sm;
  a.stages = (int)std::min<int64_t>(kMaxStages, block_smem(p.per_sm) / bytes);
  if (a.stages < 2) return p;
  a.status = ctx->ws.status;
  p.threads = threads;
  p.smem = (unsigned)(a.stages * bytes);
  return p;
}

template <auto Kernel>
void launch_ring(gc_ctx* ctx, const RmsArgs& a, const RingPlan& p, unsigned grid) {
  static uint64_t devices = 0;
  if (!allow_smem(ctx, Kernel, (int)block_smem(1), devices)) return;  // the launch's error says so
  Kernel<<<grid, p.threads + 32, p.smem, ctx->stream>>>(a);
}

template <int DT, int REGS>
void forward_ring(gc_ctx* ctx, const RmsArgs& a, const RingPlan& p, unsigned grid, bool aligned) {
  if (!aligned) launch_ring<rms_forward_ring_kernel<DT, kAnywhere, REGS>>(ctx, a, p, grid);
  else if (a.cols == (int64_t)p.threads * kCols)
    launch_ring<rms_forward_ring_kernel<DT, kFull, REGS>>(ctx, a, p, grid);
  else launch_ring<rms_forward_ring_kernel<DT, kEnds, REGS>>(ctx, a, p, grid);
}
template <int DT, bool CKPT, int REGS>
void backward_ring(gc_ctx* ctx, const RmsArgs& a, const RingPlan& p, unsigned grid, bool aligned) {
  if (!aligned) launch_ring<rms_backward_ring_kernel<DT, CKPT, kAnywhere, REGS>>(ctx, a, p, grid);
  else if (a.cols == (int64_t)p.threads * kCols)
    launch_ring<rms_backward_ring_kernel<DT, CKPT, kFull, REGS>>(ctx, a, p, grid);
  else launch_ring<rms_backward_ring_kernel<DT, CKPT, kEnds, REGS>>(ctx, a, p, grid);
}

template <int DT, bool ALIGNED>
void forward(gc_ctx* ctx, RmsArgs& a) {
  if (const RingPlan p = plan_ring(ctx, a, DT, false); p.threads) {
    LaunchScope L(ctx, GC_PHASE_RMS_FORWARD);
    const unsigned g = (unsigned)std::min<int64_t>(a.rows, (int64_t)ctx->num_sms * p.per_sm);
    if (p.regs) forward_ring<DT, kForwardRegs[1]>(ctx, a, p, g, ALIGNED);
    else forward_ring<DT, kForwardRegs[0]>(ctx, a, p, g, ALIGNED);
    return;
  }
  const Shape s = pick(ceil_div(a.row_bytes, (int64_t)16), a.rows, ctx->num_sms, 1024, 2, 1024);
  LaunchScope L(ctx, GC_PHASE_RMS_FORWARD);
  const auto kernel =
      s.wide ? rms_forward_wide_kernel<DT, ALIGNED>
      : s.warp
          ? (s.u == 1   ? rms_forward_kernel<DT, true, 1, ALIGNED>
             : s.u == 2 ? rms_forward_kernel<DT, true, 2, ALIGNED>
                        : rms_forward_kernel<DT, true, 4, ALIGNED>)
          : rms_forward_kernel<DT, false, 2, ALIGNED>;
  kernel<<<s.grid, s.threads, 0, ctx->stream>>>(a);
}

template <int DT, bool CKPT, bool ALIGNED>
gc_status backward(gc_ctx* ctx, RmsArgs& a) {
  Shape s = pick(ceil_div(a.row_bytes, (int64_t)16), a.rows, ctx->num_sms, 512, 4, 512);
  s.grid = (unsigned)std::min<int64_t>(s.grid, kMaxParts);
  const size_t smem = s.warp ? (size_t)8 * s.u * 32 * Elem<DT>::V * 4 : 0;
  if (const RingPlan p = plan_ring(ctx, a, DT, true); p.threads) {
    LaunchScope L(ctx, GC_PHASE_RMS_BACKWARD);
    s.wide = false;
    s.grid = (unsigned)std::min<int64_t>(
        {a.rows, (int64_t)ctx->num_sms * p.per_sm, kMaxParts});
    if (p.regs) backward_ring<DT, CKPT, kBackwardRegs[1]>(ctx, a, p, s.grid, ALIGNED);
    else backward_ring<DT, CKPT, kBackwardRegs[0]>(ctx, a, p, s.grid, ALIGNED);
  } else {
    LaunchScope L(ctx, GC_PHASE_RMS_BACKWARD);
    const auto kernel =
        s.wide ? rms_backward_wide_kernel<DT, CKPT, ALIGNED>
        : s.warp
            ? (s.u == 1   ? rms_backward_kernel<DT, CKPT, true, 1, ALIGNED>
               : s.u == 2 ? rms_backward_kernel<DT, CKPT, true, 2, ALIGNED>
                          : rms_backward_kernel<DT, CKPT, true, 4, ALIGNED>)
        : s.u == 2 ? rms_backward_kernel<DT, CKPT, false, 2, ALIGNED>
                   : rms_backward_kernel<DT, CKPT, false, 4, ALIGNED>;
    kernel<<<s.grid, s.threads, smem, ctx->stream>>>(a);
  }
  if (!a.dgamma || (s.grid == 1 && !s.wide)) return GC_OK;
  LaunchScope L(ctx, GC_PHASE_RMS_REDUCE);
  return launch_early(rms_reduce_kernel, dim3((unsigned)ceil_div(a.cols, (int64_t)32)), 1024, 0,
                      ctx->stream, a, (int)s.grid) == cudaSuccess
             ? GC_OK
             : GC_ERR_CUDA;
}

int64_t part_pitch(int64_t cols) { return round_up(cols, 4); }

const char* end_of(const void* p, int64_t rows, int64_t ld, int64_t cols, int dtype) {
  return static_cast<const char*>(p) + ((rows - 1) * ld + cols) * elem_size(dtype);
}

}  // namespace

int64_t rms_scratch_bytes(int64_t rows, int64_t cols) {
  return std::min(rows, kMaxParts) * part_pitch(cols) * 4;
}

gc_status launch_rms_forward(gc_ctx* ctx, const void* x, int64_t ldx, const void* res,
                             int64_t ldres, int dtype, int64_t rows, int64_t cols,
                             const void* gamma, int ptype, float eps, void* h, int64_t ldh,
                             void* y, int64_t ldy, float* rstd, uint8_t* codes, uint8_t* scales,
                             uint8_t* y_codes, uint8_t* y_scales) {
  if (rows == 0 || cols == 0) return GC_OK;
  const int64_t e = elem_size(dtype);
  RmsArgs a{};
  a.x = static_cast<const char*>(x);
  a.res = static_cast<const char*>(res);
  a.xend = end_of(x, rows, ldx, cols, dtype);
  if (res) a.resend = end_of(res, rows, ldres, cols, dtype);
  a.h = static_cast<char*>(h);
  a.y = static_cast<char*>(y);
  a.gamma = gamma;
  a.ptype = ptype;
  a.eps = eps;
  a.rstd = rstd;
  a.codes = codes;
  a.scales = scales;
  a.ycodes = y_codes;
  a.yscales = y_scales;
  a.rows = rows;
  a.cols = cols;
  a.row_bytes = cols * e;
  a.xpitch = ldx * e;
  a.respitch = ldres * e;
  a.hpitch = ldh * e;
  a.ypitch = ldy * e;
  a.codes_pitch = ckpt_codes_pitch(cols);
  a.scales_pitch = ckpt_scales_pitch(cols);
  const bool al = rows == 1 || (row_aligned(ldx, dtype) && (!res || row_aligned(ldres, dtype)) &&
                                (!h || row_aligned(ldh, dtype)) && (!y || row_aligned(ldy, dtype)));
  if (dtype == GC_F32) al ? forward<GC_F32, true>(ctx, a) : forward<GC_F32, false>(ctx, a);
  else if (dtype == GC_BF16) al ? forward<GC_BF16, true>(ctx, a) : forward<GC_BF16, false>(ctx, a);
  else al ? forward<GC_F16, true>(ctx, a) : forward<GC_F16, false>(ctx, a);
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

gc_status launch_rms_backward(gc_ctx* ctx, const void* dy, int64_t lddy, const void* dres,
                              int64_t lddres, const void* h, int64_t ldh, const uint8_t* codes,
                              const uint8_t* scales, int dtype, int64_t rows, int64_t cols,
                              const void* gamma, int ptype, const float* rstd, void* dx,
                              int64_t lddx, float* dgamma, int accumulate, float* part) {
  if (cols == 0) return GC_OK;
  if (rows == 0) {
    if (!dgamma || accumulate) return GC_OK;
    return cudaMemsetAsync(dgamma, 0, cols * 4, ctx->stream) == cudaSuccess ? GC_OK : GC_ERR_CUDA;
  }
  const int64_t e = elem_size(dtype);
  RmsArgs a{};
  a.dy = static_cast<const char*>(dy);
  a.dyend = end_of(dy, rows, lddy, cols, dtype);
  a.dres = static_cast<const char*>(dres);
  if (dres) a.dresend = end_of(dres, rows, lddres, cols, dtype);
  a.x = static_cast<const char*>(h);
  if (h) a.xend = end_of(h, rows, ldh, cols, dtype);
  a.y = static_cast<char*>(dx);
  a.gamma = gamma;
  a.ptype = ptype;
  a.rstd = const_cast<float*>(rstd);
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  a.dgamma = dgamma;
  a.part = part;
  a.part_pitch = part_pitch(cols);
  a.accumulate = accumulate;
  a.rows = rows;
  a.cols = cols;
  a.row_bytes = cols * e;
  a.dypitch = lddy * e;
  a.drespitch = lddres * e;
  a.xpitch = ldh * e;
  a.ypitch = lddx * e;
  a.codes_pitch = ckpt_codes_pitch(cols);
  a.scales_pitch = ckpt_scales_pitch(cols);
  const bool al =
      rows == 1 || (row_aligned(lddy, dtype) && (!dres || row_aligned(lddres, dtype)) &&
                    (!h || row_aligned(ldh, dtype)) && row_aligned(lddx, dtype));
  gc_status st = GC_OK;
  auto go = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (codes) st = al ? backward<DT, true, true>(ctx, a) : backward<DT, true, false>(ctx, a);
    else st = al ? backward<DT, false, true>(ctx, a) : backward<DT, false, false>(ctx, a);
  };
  if (dtype == GC_F32) go(std::integral_constant<int, GC_F32>{});
  else if (dtype == GC_BF16) go(std::integral_constant<int, GC_BF16>{});
  else go(std::integral_constant<int, GC_F16>{});
  if (st != GC_OK) return st;
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

}  // namespace gc
