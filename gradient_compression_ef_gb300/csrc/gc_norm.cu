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
// A row lives in the registers of the threads that own it, so each input is
// read once: the mean, then the centred sum of squares (no cancellation),
// then the output.  All sums are fp32, in an order that sizes alone decide.
// Both passes are bound by memory; what they need is loads in flight and few
// instructions per element:
//   cols <= 512         a warp per row, up to 4 units of 16 bytes per lane;
//   up to 16384 columns a block walks over rows that bulk copies bring into a
//   (backward 8192),    ring of stages in shared memory, several rows ahead; a
//   while two rows fit  thread owns 16 columns of all rows, the column sums
//   in shared memory    stay in its registers, and nothing but the stage
//                       changes from row to row;
//   wider still         the row is read again from L2 for each of its passes.
// The backward pass leaves one partial row of column sums per block; a second
// small grid adds the partials in block order.
//
// Measured, bytes read and written once over the time (a plain copy: 6.77
// TB/s), forward and backward with a checkpoint: 16384 x 4096 bf16 74 us (4.5
// TB/s) and 84 (4.0), fp32 104 (5.8) and 111 (5.5); without one bf16
// 55 (4.9) and 82 (4.9), fp32 92 (5.8) and 130 (6.2).  fp32 is near the memory
// rate; 16-bit rows have twice the elements per byte, and are held up by
// instruction issue (25 per element and lane forward) and shared-memory latency
// at the 20 to 24 warps per SM that registers allow.  Rows on odd boundaries: 16001 x 4099 fp32
// without a checkpoint 119 us (4.4) and 196 (4.0), bf16 with one 140 and 137
// (2.4).  Narrow rows: 65536 x 500 bf16 57 (2.9) and 116 (1.4).  Wider than the
// ring: 4096 x 20000 bf16 210 (2.0) and 136 (3.0).  The column sums' second grid
// 8 us at 4096 columns.
#include <algorithm>

#include "gc_rows.cuh"

namespace gc {
namespace {

struct NormArgs {
  const char *x, *dy;        // input (forward; backward without a checkpoint)
  const char *xend, *dyend;  // the matrices' ends
  char* out;                 // y or dx
  const void *gamma, *beta;
  float *mean, *rstd;
  uint8_t *codes, *scales;
  float *dgamma, *dbeta;  // gradients, or NULL
  float* part;            // [parts][2][cols]
  int64_t rows, cols, row_bytes, xpitch, dypitch, outpitch, codes_pitch, scales_pitch;
  float eps;
  int ptype, accumulate;
  // ring of stages (set at launch)
  uint32_t* status;
  uint32_t second_at, scales_at, stage_bytes;  // within a stage: x or codes; scale bytes
  int stages;
};

// A row per warp, K units per lane, no barrier; gamma and beta lie in shared
// memory, shared by the block's warps.
template <int DT, int K, bool ALIGNED>
__global__ void __launch_bounds__(256, 4)
    norm_forward_warp_kernel(const __grid_constant__ NormArgs a) {
  using L = Elem<DT>;
  constexpr int V = L::V, H = V / 2;
  extern __shared__ __align__(16) float params[];  // gamma, beta: [2][K * 32 * V]
  for (int c = threadIdx.x * V; c < K * 32 * V; c += 256 * V) {
    float v[V];
    load_params<V>(v, a.gamma, a.ptype, c, a.cols, 1.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) params[c + j] = v[j];
    load_params<V>(v, a.beta, a.ptype, c, a.cols, 0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) params[K * 32 * V + c + j] = v[j];
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const uint32_t gam = sm100::smem_u32(params) + lane * (V * 4), bet = gam + K * 32 * V * 4;
  const float inv_n = 1.0f / (float)a.cols;
  const bool inner = K * 512 + (ALIGNED ? 0 : 16) <= a.row_bytes;
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < a.rows;
       row += (int64_t)gridDim.x * 8) {
    uint4 raw[K];
    load_run<DT, ALIGNED>(raw, a.x + row * a.xpitch, 0u, inner, a.row_bytes, a.xend);
    float2 s = both(0.0f);
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float2 v[H];
      unpack2<DT>(raw[i], v);
#pragma unroll
      for (int j = 0; j < H; ++j) s = __fadd2_rn(s, v[j]);
    }
    const float mean = warp_allsum(s.x + s.y) * inv_n;
    const float2 m = both(-mean);
    s = both(0.0f);
#pragma unroll
    for (int i = 0; i < K; ++i) {
      keep_packed(raw[i]);
      float2 v[H];
      unpack2<DT>(raw[i], v);
#pragma unroll
      for (int j = 0; j < H; ++j) v[j] = __fadd2_rn(v[j], m);
      if (!inner) {
        const int64_t left = a.row_bytes - (i * 32 + lane) * 16;
#pragma unroll
        for (int j = 0; j < H; ++j) {
          if (2 * j * elem_size(DT) >= left) v[j].x = 0.0f;
          if ((2 * j + 1) * elem_size(DT) >= left) v[j].y = 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < H; ++j) s = __ffma2_rn(v[j], v[j], s);
    }
    const float rstd = rsqrtf(warp_allsum(s.x + s.y) * inv_n + a.eps);
    if (lane == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    const float2 rs = both(rstd);
    uint8_t* codes = a.codes + row * a.codes_pitch + lane * V;
    uint8_t* scales = a.scales + row * a.scales_pitch + lane * V / kActGroup;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      keep_packed(raw[i]);
      if (a.codes) {
        float f[V];
        L::unpack(raw[i], f);
        const uint32_t sb = scale_byte(group_max_bits<DT>(raw[i]));
        if (inner || (i * 32 + lane) * V < a.codes_pitch) {
          store_codes<DT>(codes + i * 32 * V, raw[i], f, sb);
          if (lane % (kActGroup / V) == 0) scales[i * 32 * V / kActGroup] = (uint8_t)sb;
        }
      }
      float2 v[H], g[H], b[H];
      unpack2<DT>(raw[i], v);
      lds_params<V>(g, gam + i * 32 * V * 4);
      lds_params<V>(b, bet + i * 32 * V * 4);
#pragma unroll
      for (int j = 0; j < H; ++j)
        v[j] = __ffma2_rn(__fmul2_rn(__fadd2_rn(v[j], m), rs), g[j], b[j]);
      raw[i] = pack2<DT>(v);
    }
    store_run<DT, ALIGNED>(a.out + row * a.outpitch, 0u, inner, a.row_bytes, raw);
  }
}

// A row per block, one unit per thread (few rows: the shortest way through),
// or K == 0: rows wider than the other kernels hold, read again (from L2) for
// each of the three passes.
template <int DT, int K, bool ALIGNED>
__global__ void __launch_bounds__(1024)
    norm_forward_kernel(const __grid_constant__ NormArgs a) {
  using E = Elem<DT>;
  constexpr int V = E::V, KK = K ? K : 1;
  __shared__ float2 slot[2][32];
  RowSum<false> sum{slot};
  const int nt = blockDim.x, t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const float inv_n = 1.0f / (float)a.cols;
  const int loops = K ? K : (int)((a.codes_pitch / V + nt - 1) / nt);
  const char* x = a.x + row * a.xpitch;
  uint4 raw[KK];
  auto off = [&](int i) { return ((int64_t)t + (int64_t)i * nt) * 16; };
  auto load = [&](int i) { return load_unit<DT, ALIGNED>(x, off(i), a.row_bytes, a.xend); };
  if (K) {
#pragma unroll
    for (int i = 0; i < KK; ++i) raw[i] = load(i);
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < (K ? K : loops); ++i) {
    float v[V];
    E::unpack(K ? raw[K ? i : 0] : load(i), v);
#pragma unroll
    for (int j = 0; j < V; ++j) s += v[j];
  }
  const float mean = sum(s) * inv_n;
  if (K) {
#pragma unroll
    for (int i = 0; i < KK; ++i) keep_packed(raw[i]);
  }
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < (K ? K : loops); ++i) {
    float v[V];
    E::unpack(K ? raw[K ? i : 0] : load(i), v);
    const int64_t left = a.cols - off(i) / elem_size(DT);
    if (left >= V) {
#pragma unroll
      for (int j = 0; j < V; ++j) q = fmaf(v[j] - mean, v[j] - mean, q);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j < left) q = fmaf(v[j] - mean, v[j] - mean, q);
    }
  }
  const float rstd = rsqrtf(sum(q) * inv_n + a.eps);
  if (t == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < (K ? K : loops); ++i) {
    float v[V], g[V], b[V];
    if (K) keep_packed(raw[K ? i : 0]);
    E::unpack(K ? raw[K ? i : 0] : load(i), v);
    const int64_t c = off(i) / elem_size(DT);
    if (a.codes) {
      const uint4 r = K ? raw[K ? i : 0] : load(i);
      const uint32_t sb = scale_byte(group_max_bits<DT>(r));
      if (c < a.codes_pitch) {
        store_codes<DT>(a.codes + row * a.codes_pitch + c, r, v, sb);
        if (t % (kActGroup / V) == 0)
          a.scales[row * a.scales_pitch + c / kActGroup] = (uint8_t)sb;
      }
    }
    load_params<V>(g, a.gamma, a.ptype, c, a.cols, 1.0f);
    load_params<V>(b, a.beta, a.ptype, c, a.cols, 0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = fmaf((v[j] - mean) * rstd, g[j], b[j]);
    store_unit<DT, ALIGNED>(a.out + row * a.outpitch, off(i), a.row_bytes, E::pack(v));
  }
}

// A block's column sums go to its partial row, or, when it is the only block,
// to the gradients.
__device__ __forceinline__ void put_sums(const NormArgs& a, int64_t part, bool only, int64_t c,
                                         float g, float b) {
  if (!only) {
    a.part[part * 2 * a.cols + c] = g;
    a.part[(part * 2 + 1) * a.cols + c] = b;
    return;
  }
  if (a.dgamma) a.dgamma[c] = a.accumulate ? a.dgamma[c] + g : g;
  if (a.dbeta) a.dbeta[c] = a.accumulate ? a.dbeta[c] + b : b;
}

// A unit's inputs as they lie in memory.
template <int DT, bool CKPT>
struct RawUnit {
  uint4 dy, x;
};
template <int DT>
struct RawUnit<DT, true> {
  uint4 dy;
  Codes<Elem<DT>::V> c;
  uint32_t b;
};

template <int DT, bool CKPT, bool ALIGNED>
__device__ __forceinline__ void load_raw(RawUnit<DT, CKPT>& r, const NormArgs& a, int64_t row,
                                         int64_t off) {
  constexpr int V = Elem<DT>::V;
  const bool whole = ALIGNED && off + 16 <= a.row_bytes;
  const char* dy = a.dy + row * a.dypitch;
  r.dy = whole ? __ldg(reinterpret_cast<const uint4*>(dy + off))
               : load_unit<DT, ALIGNED>(dy, off, a.row_bytes, a.dyend);
  if constexpr (CKPT) {
    const int64_t c = off / elem_size(DT);
    r.c = Codes<V>{};
    r.b = 0u;
    if (c < a.codes_pitch) {
      r.c = load_codes<V>(a.codes + row * a.codes_pitch + c);
      r.b = __ldg(a.scales + row * a.scales_pitch + c / kActGroup);
    }
  } else {
    const char* x = a.x + row * a.xpitch;
    r.x = whole ? __ldg(reinterpret_cast<const uint4*>(x + off))
                : load_unit<DT, ALIGNED>(x, off, a.row_bytes, a.xend);
  }
}

template <int DT, bool CKPT>
__device__ __forceinline__ void unpack_raw(const RawUnit<DT, CKPT>& r, float (&dy)[Elem<DT>::V],
                                           float (&x)[Elem<DT>::V]) {
  Elem<DT>::unpack(r.dy, dy);
  if constexpr (CKPT) decode<Elem<DT>::V>(x, r.c, r.b);
  else Elem<DT>::unpack(r.x, x);
}

// A row per warp at a time, K units per lane, the next row's loads issued
// before the current row's sums; the column sums in registers over the
// warp's rows.
template <int DT, int K, bool CKPT, bool ALIGNED>
__global__ void __launch_bounds__(256, 2)
    norm_backward_kernel(const __grid_constant__ NormArgs a) {
  using E = Elem<DT>;
  constexpr int V = E::V;
  RowSum<true> sum{nullptr};
  constexpr int nt = 32;
  const int t = threadIdx.x & 31, per_block = blockDim.x / 32;
  const int64_t step = (int64_t)gridDim.x * per_block;
  int64_t row = (int64_t)blockIdx.x * per_block + (threadIdx.x >> 5);
  const float inv_n = 1.0f / (float)a.cols;
  auto off = [&](int i) { return ((int64_t)t + (int64_t)i * nt) * 16; };
  float sg[K][V], sb[K][V];
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) sg[i][j] = sb[i][j] = 0.0f;

  RawUnit<DT, CKPT> next[K];
  float mean_n = 0.0f, rstd_n = 0.0f;
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < K; ++i) load_raw<DT, CKPT, ALIGNED>(next[i], a, r, off(i));
    mean_n = __ldg(a.mean + r);
    rstd_n = __ldg(a.rstd + r);
  };
  if (row < a.rows) fetch(row);
  for (; row < a.rows; row += step) {
    float d[K][V], n[K][V];
    const float mean = mean_n, rstd = rstd_n;
#pragma unroll
    for (int i = 0; i < K; ++i) unpack_raw<DT, CKPT>(next[i], d[i], n[i]);
    if (row + step < a.rows) fetch(row + step);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float g[V];
      load_params<V>(g, a.gamma, a.ptype, off(i) / elem_size(DT), a.cols, 1.0f);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        n[i][j] = (n[i][j] - mean) * rstd;
        sg[i][j] = fmaf(d[i][j], n[i][j], sg[i][j]);
        sb[i][j] += d[i][j];
        d[i][j] *= g[j];  // dy is 0 past the last column
        s1 += d[i][j];
        s2 = fmaf(d[i][j], n[i][j], s2);
      }
    }
    const float2 c12 = sum(s1, s2);
    const float c1 = c12.x * inv_n, c2 = c12.y * inv_n;
#pragma unroll
    for (int i = 0; i < K; ++i) {
#pragma unroll
      for (int j = 0; j < V; ++j) d[i][j] = rstd * (d[i][j] - c1 - n[i][j] * c2);
      store_unit<DT, ALIGNED>(a.out + row * a.outpitch, off(i), a.row_bytes, E::pack(d[i]));
    }
  }

  if (!a.dgamma && !a.dbeta) return;
  // the block's warps own the same columns: add them in warp order
  extern __shared__ float acc[];  // [2][codes_pitch]
  const int w8 = (int)a.codes_pitch;
  for (int w = 0; w < per_block; ++w) {
    if ((int)(threadIdx.x >> 5) == w) {
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const int c = (t + i * 32) * V;
        if (c < w8) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            acc[c + j] = (w ? acc[c + j] : 0.0f) + sg[i][j];
            acc[w8 + c + j] = (w ? acc[w8 + c + j] : 0.0f) + sb[i][j];
          }
        }
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < a.cols; c += blockDim.x)
    put_sums(a, blockIdx.x, gridDim.x == 1, c, acc[c], acc[w8 + c]);
}

// ---------------------------------------------------------------------------
// Rows through a ring of stages in shared memory.
// ---------------------------------------------------------------------------
constexpr int kMaxStages = 6;
constexpr int kCols = 16;  // columns per thread

// One thread's part: row `row` into a stage.  BACK: dy, then x or the
// checkpoint; else x.
template <int DT, bool BACK, bool CKPT>
__device__ __forceinline__ void fill_stage(const NormArgs& a, int64_t row, char* stage,
                                           uint64_t* full) {
  using namespace sm100;
  const char* r0 = BACK ? a.dy + row * a.dypitch : a.x + row * a.xpitch;
  const uint32_t n0 = bulk_size<DT>(r0, a.row_bytes, BACK ? a.dyend : a.xend, stage);
  const char* r1 = a.x + row * a.xpitch;
  uint32_t n1 = 0, n2 = 0;
  if (BACK) {
    if (CKPT) {
      n1 = (uint32_t)a.codes_pitch;
      n2 = (uint32_t)a.scales_pitch;
    } else {
      n1 = bulk_size<DT>(r1, a.row_bytes, a.xend, stage + a.second_at);
    }
  }
  mbar_arrive_expect_tx(full, n0 + n1 + n2);
  if (n0) bulk_load(stage, r0 - (reinterpret_cast<uintptr_t>(r0) & 15u), n0, full);
  if (BACK) {
    if (CKPT) {
      bulk_load(stage + a.second_at, a.codes + row * a.codes_pitch, n1, full);
      bulk_load(stage + a.scales_at, a.scales + row * a.scales_pitch, n2, full);
    } else if (n1) {
      bulk_load(stage + a.second_at, r1 - (reinterpret_cast<uintptr_t>(r1) & 15u), n1, full);
    }
  }
}

// The backward kernel's producer warp: copies the block's rows, stage after
// stage, as the row's warps hand the stages back.  (The copies' address
// arithmetic, done by a thread of the row's warps between two barriers, kept
// all of them waiting: 16384 x 4096 bf16 88 -> 82 us.  The forward kernel
// copies half as much and does without: its extra warp would cost one of the
// four blocks that an SM's registers hold, 74 -> 83 us.)
template <int DT, bool CKPT>
__device__ __forceinline__ bool produce(const NormArgs& a, char* stages, uint64_t* full,
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
      fill_stage<DT, true, CKPT>(a, row, stages + ring.st * a.stage_bytes, &full[ring.st]);
    }
  }
  return ok;
}

// kCols columns per thread; a warp's units are consecutive, lane l having
// units l, l + 32, ... of them.
// Registers decide how many warps an SM holds, and these kernels live from
// that: gamma and beta (read by each thread at its own place) are kept in
// shared memory, a row between its passes packed as it came.  64, 80
// and 96 registers give 8, 6 and 5 warps per scheduler.
constexpr int kBackwardRegs = 96;
constexpr int kBackwardWarps = 20;  // per SM
constexpr int forward_regs(int rows) { return rows == 2 ? 80 : 64; }
constexpr int forward_warps(int rows) { return rows == 2 ? 24 : 32; }  // per SM
// Rows that a block of the forward kernel has in hand at once: 16-bit rows go
// two at a time where one block's registers hold two.  The sums over its warps
// (about 1000 cycles each, most of it waiting for the slowest warp) are then
// paid once for both: 6000 x 11008 bf16 took 111 us by one row at a time, 96
// by two; 16384 x 4096 without a checkpoint 66 and 54.
int forward_rows(int64_t codes_pitch, int dtype) {
  return dtype != GC_F32 && codes_pitch <= forward_warps(2) * 32 * kCols ? 2 : 1;
}

template <int V>
__device__ __forceinline__ void sts_params(uint32_t at, const void* p, int ptype, int64_t c,
                                           int64_t cols, float fill) {
  float v[V];
  load_params<V>(v, p, ptype, c, cols, fill);
#pragma unroll
  for (int j = 0; j < V; j += 4)
    sm100::sts128(at + j * 4, make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]));
}

template <int DT, int R, int ROWS>
__global__ void __maxnreg__(forward_regs(R))
    norm_forward_ring_kernel(const __grid_constant__ NormArgs a) {
  using namespace sm100;
  using L = Elem<DT>;
  constexpr int V = L::V, K = kCols / V, H = V / 2;
  extern __shared__ __align__(128) char stages[];
  __shared__ __align__(16) float slot[2][36 * R];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  const int t = threadIdx.x, nt = blockDim.x;
  for (int i = t; i < 72 * R; i += nt) slot[i / (36 * R)][i % (36 * R)] = 0.0f;
  int64_t fetch = blockIdx.x;  // next row to copy (thread 0)
  if (t == 0) {
    for (int i = 0; i < a.stages; ++i) mbar_init(&full[i], 1);
    mbar_fence_init();
    for (int i = 0; i < a.stages && fetch < a.rows; ++i, fetch += gridDim.x)
      fill_stage<DT, false, false>(a, fetch, stages + i * a.stage_bytes, &full[i]);
  }
  __syncthreads();
  RowsSum<R> sum{slot, nt};
  const uint32_t u0 = (t & ~31) * K, u1 = u0 + (t & 31);  // the warp's and the thread's first unit
  const uint32_t base = smem_u32(stages) + u1 * 16;
  const float inv_n = 1.0f / (float)a.cols;
  // the thread's own gamma, then beta, behind the stages
  const uint32_t gam = smem_u32(stages) + a.stages * a.stage_bytes + u1 * (V * 4);
  const uint32_t bet = gam + nt * (kCols * 4);
  int left[K];  // bytes of the row from the unit on
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int64_t u = u1 + i * 32;
    left[i] = (int)max((int64_t)0, min((int64_t)16, a.row_bytes - u * 16));
    sts_params<V>(gam + i * 32 * (V * 4), a.gamma, a.ptype, u * V, a.cols, 1.0f);
    sts_params<V>(bet + i * 32 * (V * 4), a.beta, a.ptype, u * V, a.cols, 0.0f);
  }
  bool ok = true;
  RingPos ring;
  const int64_t hop = gridDim.x;
  for (int64_t row = blockIdx.x; row < a.rows; row += R * hop) {
    uint4 raw[R][K];
    float s[R];
    RingPos next = ring;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool here = r == 0 || row + r * hop < a.rows;
      float2 c = both(0.0f);
      if (here && !mbar_wait(&full[next.st], next.ph, kWaitCycles)) ok = false;
      const uint32_t stage = base + next.st * a.stage_bytes;
      const uint32_t mis =
          ROWS == kAnywhere
              ? (uint32_t)(reinterpret_cast<uintptr_t>(a.x + (row + r * hop) * a.xpitch) & 15u)
              : 0u;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        raw[r][i] = make_uint4(0u, 0u, 0u, 0u);
        if (here && (ROWS == kFull || left[i] > 0))
          raw[r][i] = staged_unit<DT, ROWS>(stage + i * 512, mis, left[i]);
        float2 v[H];
        unpack2<DT>(raw[r][i], v);
#pragma unroll
        for (int j = 0; j < H; ++j) c = __fadd2_rn(c, v[j]);
      }
      s[r] = c.x + c.y;
      if (here) next.next(a.stages);
    }
    sum(s, ok);
    if (!ok) break;
    // every thread holds its part of the rows: their stages take later ones
    if (t == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (fetch >= a.rows) break;
        fence_proxy_async_smem();
        fill_stage<DT, false, false>(a, fetch, stages + ring.st * a.stage_bytes, &full[ring.st]);
        fetch += hop;
        ring.next(a.stages);
      }
    }
    ring = next;
    float mean[R], q[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = s[r] * inv_n;
      const float2 m = both(-mean[r]);
      float2 c = both(0.0f);
#pragma unroll
      for (int i = 0; i < K; ++i) {
        keep_packed(raw[r][i]);
        float2 v[H];
        unpack2<DT>(raw[r][i], v);
#pragma unroll
        for (int j = 0; j < H; ++j) v[j] = __fadd2_rn(v[j], m);
        if (ROWS != kFull && left[i] < 16) {
#pragma unroll
          for (int j = 0; j < H; ++j) {
            if (2 * j * elem_size(DT) >= left[i]) v[j].x = 0.0f;
            if ((2 * j + 1) * elem_size(DT) >= left[i]) v[j].y = 0.0f;
          }
        }
#pragma unroll
        for (int j = 0; j < H; ++j) c = __ffma2_rn(v[j], v[j], c);
      }
      q[r] = c.x + c.y;
    }
    sum(q, ok);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t at = row + r * hop;
      if (r > 0 && at >= a.rows) break;
      const float rstd = rsqrtf(q[r] * inv_n + a.eps);
      if (t == 0) {
        a.mean[at] = mean[r];
        a.rstd[at] = rstd;
      }
      const float2 m = both(-mean[r]), rs = both(rstd);
      uint8_t* codes = a.codes + at * a.codes_pitch;
      uint8_t* scales = a.scales + at * a.scales_pitch;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        keep_packed(raw[r][i]);
        const uint32_t u = u1 + i * 32;
        if (a.codes) {
          float f[V];
          L::unpack(raw[r][i], f);
          const uint32_t sb = scale_byte(group_max_bits<DT>(raw[r][i]));
          if (ROWS == kFull || u * V < a.codes_pitch) {
            store_codes<DT>(codes + u * V, raw[r][i], f, sb);
            if (t % (kActGroup / V) == 0) scales[u * V / kActGroup] = (uint8_t)sb;
          }
        }
        float2 v[H], g[H], b[H];
        unpack2<DT>(raw[r][i], v);
        lds_params<V>(g, gam + i * 32 * (V * 4));
        lds_params<V>(b, bet + i * 32 * (V * 4));
#pragma unroll
        for (int j = 0; j < H; ++j)
          v[j] = __ffma2_rn(__fmul2_rn(__fadd2_rn(v[j], m), rs), g[j], b[j]);
        raw[r][i] = pack2<DT>(v);
      }
      put_units<DT, ROWS>(a.out + at * a.outpitch, u0, a.row_bytes, raw[r]);
    }
  }
  ring_end(ok, a.status);
}

// A thread's part of a row between the two passes, packed: dy, and x or (from
// a checkpoint) the restored values as bf16, which holds them exactly.
template <int DT, bool CKPT>
struct Packed {
  uint4 dy, x;
};
template <>
struct Packed<GC_F32, true> {
  uint4 dy;
  uint2 x;
};

template <int DT, bool CKPT>
__device__ __forceinline__ void unpack_x(const Packed<DT, CKPT>& p, float2 (&v)[Elem<DT>::V / 2]) {
  if constexpr (CKPT) {
    uint32_t w[Elem<DT>::V / 2];
    w[0] = p.x.x;
    w[1] = p.x.y;
    if constexpr (DT != GC_F32) {
      w[2] = p.x.z;
      w[3] = p.x.w;
    }
#pragma unroll
    for (int j = 0; j < Elem<DT>::V / 2; ++j)
      v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  } else {
    unpack2<DT>(p.x, v);
  }
}

// Row sums s1 = sum(d), s2 = sum(d (x - mean)), with d = dy gamma; then
//   dx = rstd d - (s2 rstd^3 / n) (x - mean) - s1 rstd / n.
template <int DT, bool CKPT, int ROWS>
__global__ void __maxnreg__(kBackwardRegs)
    norm_backward_ring_kernel(const __grid_constant__ NormArgs a) {
  using namespace sm100;
  constexpr int V = Elem<DT>::V, K = kCols / V, H = V / 2;
  extern __shared__ __align__(128) char stages[];
  __shared__ __align__(16) float slot[2][36 * 2];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  const int t = threadIdx.x, nt = blockDim.x - 32;  // the last warp is the producer
  for (int i = t; i < 72 * 2; i += blockDim.x) slot[i / (36 * 2)][i % (36 * 2)] = 0.0f;
  if (t == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], nt / 32);
    }
    mbar_fence_init();
  }
  __syncthreads();
  if (t >= nt) {
    ring_end(produce<DT, CKPT>(a, stages, full, empty), a.status);
    return;
  }
  RowsSum<2> sum{slot, nt};
  const uint32_t base = smem_u32(stages);
  const uint32_t u0 = (t & ~31) * K, u1 = u0 + (t & 31);  // the warp's and the thread's first unit
  const uint32_t gam = base + a.stages * a.stage_bytes + u1 * (V * 4);  // the thread's own gamma
  const float inv_n = 1.0f / (float)a.cols;
  float2 sg[K][H], sb[K][H];
  int left[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int64_t u = u1 + i * 32;
    left[i] = (int)max((int64_t)0, min((int64_t)16, a.row_bytes - u * 16));
    sts_params<V>(gam + i * 32 * (V * 4), a.gamma, a.ptype, u * V, a.cols, 1.0f);
#pragma unroll
    for (int j = 0; j < H; ++j) sg[i][j] = sb[i][j] = both(0.0f);
  }
  const int64_t hop = gridDim.x;
  const char *dyp = a.dy + blockIdx.x * a.dypitch, *xp = a.x + blockIdx.x * a.xpitch;
  char* out = a.out + blockIdx.x * a.outpitch;
  float mean = 0.0f, rstd = 0.0f;
  if (blockIdx.x < a.rows) {
    mean = __ldg(a.mean + blockIdx.x);
    rstd = __ldg(a.rstd + blockIdx.x);
  }
  bool ok = true;
  RingPos ring;
  for (int64_t row = blockIdx.x; row < a.rows;
       row += hop, dyp += hop * a.dypitch, xp += hop * a.xpitch, out += hop * a.outpitch) {
    float mean_n = 0.0f, rstd_n = 0.0f;
    if (row + hop < a.rows) {
      mean_n = __ldg(a.mean + row + hop);
      rstd_n = __ldg(a.rstd + row + hop);
    }
    ok = mbar_wait(&full[ring.st], ring.ph, kWaitCycles);
    const uint32_t stage = base + ring.st * a.stage_bytes;
    const uint32_t mis0 =
        ROWS == kAnywhere ? (uint32_t)(reinterpret_cast<uintptr_t>(dyp) & 15u) : 0u;
    const uint32_t mis1 =
        ROWS == kAnywhere ? (uint32_t)(reinterpret_cast<uintptr_t>(xp) & 15u) : 0u;
    const float2 m = both(-mean), rs = both(rstd);
    Packed<DT, CKPT> in[K];
    float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const uint32_t u = u1 + i * 32;
      in[i] = Packed<DT, CKPT>{};
      if (ROWS != kFull && left[i] <= 0) continue;
      in[i].dy = staged_unit<DT, ROWS>(stage + u * 16, mis0, left[i]);
      if constexpr (CKPT) {
        const uint32_t at = stage + a.second_at + u * V;
        const uint32_t b = lds_u8(stage + a.scales_at + u / (kActGroup / V)) * 0x00800080u;
        const uint32_t c0 = lds_u32(at);
        in[i].x.x = decode2(c0, 0x1100u, b);
        in[i].x.y = decode2(c0, 0x3322u, b);
        if constexpr (DT != GC_F32) {
          const uint32_t c1 = lds_u32(at + 4);
          in[i].x.z = decode2(c1, 0x1100u, b);
          in[i].x.w = decode2(c1, 0x3322u, b);
        }
      } else {
        in[i].x = staged_unit<DT, ROWS>(stage + a.second_at + u * 16, mis1, left[i]);
      }
      float2 d[H], n[H], g[H];
      unpack2<DT>(in[i].dy, d);
      unpack_x<DT, CKPT>(in[i], n);
      lds_params<V>(g, gam + i * 32 * (V * 4));
#pragma unroll
      for (int j = 0; j < H; ++j) {
        n[j] = __fadd2_rn(n[j], m);
        sg[i][j] = __ffma2_rn(__fmul2_rn(d[j], rs), n[j], sg[i][j]);
        sb[i][j] = __fadd2_rn(sb[i][j], d[j]);
        d[j] = __fmul2_rn(d[j], g[j]);  // dy is 0 past the last column
        s1 = __fadd2_rn(s1, d[j]);
        s2 = __ffma2_rn(d[j], n[j], s2);
      }
    }
    // the warp holds its part of the row
    __syncwarp();
    if ((t & 31) == 0) mbar_arrive(&empty[ring.st]);
    ring.next(a.stages);
    float s[2] = {s1.x + s1.y, s2.x + s2.y};
    sum(s, ok);
    if (!ok) break;
    const float2 c1 = both(-s[0] * inv_n * rstd);
    const float2 c2 = both(-s[1] * inv_n * rstd * rstd * rstd);
    uint4 res[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      keep_packed(in[i].dy);
      float2 d[H], n[H], g[H];
      unpack2<DT>(in[i].dy, d);
      unpack_x<DT, CKPT>(in[i], n);
      lds_params<V>(g, gam + i * 32 * (V * 4));
#pragma unroll
      for (int j = 0; j < H; ++j)
        d[j] = __ffma2_rn(__fmul2_rn(d[j], g[j]), rs, __ffma2_rn(__fadd2_rn(n[j], m), c2, c1));
      res[i] = pack2<DT>(d);
    }
    put_units<DT, ROWS>(out, u0, a.row_bytes, res);
    mean = mean_n;
    rstd = rstd_n;
  }
  ring_end(ok, a.status);

  if (!a.dgamma && !a.dbeta) return;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int64_t c = (int64_t)(u1 + i * 32) * V;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (c + j < a.cols)
        put_sums(a, blockIdx.x, gridDim.x == 1, c + j, j & 1 ? sg[i][j / 2].y : sg[i][j / 2].x,
                 j & 1 ? sb[i][j / 2].y : sb[i][j / 2].x);
  }
}

// Rows wider than a block's registers hold: dx by a block per row that reads
// the row twice (the second time from L2), the column sums by a grid of its
// own.
template <int DT, bool CKPT, bool ALIGNED>
__global__ void __launch_bounds__(512)
    norm_backward_wide_kernel(const __grid_constant__ NormArgs a) {
  using E = Elem<DT>;
  constexpr int V = E::V;
  __shared__ float2 slot[2][32];
  RowSum<false> sum{slot};
  const int loops = (int)((a.codes_pitch / V + blockDim.x - 1) / blockDim.x);
  const int64_t row = blockIdx.x;
  const float inv_n = 1.0f / (float)a.cols, mean = a.mean[row], rstd = a.rstd[row];
  auto fetch = [&](int i, float (&d)[V], float (&n)[V]) {
    const int64_t off = ((int64_t)threadIdx.x + (int64_t)i * blockDim.x) * 16;
    RawUnit<DT, CKPT> r;
    load_raw<DT, CKPT, ALIGNED>(r, a, row, off);
    unpack_raw<DT, CKPT>(r, d, n);
    float g[V];
    load_params<V>(g, a.gamma, a.ptype, off / elem_size(DT), a.cols, 1.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      n[j] = (n[j] - mean) * rstd;
      d[j] *= g[j];
    }
    return off;
  };
  float s1 = 0.0f, s2 = 0.0f;
  for (int i = 0; i < loops; ++i) {
    float d[V], n[V];
    fetch(i, d, n);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s1 += d[j];
      s2 = fmaf(d[j], n[j], s2);
    }
  }
  const float2 c12 = sum(s1, s2);
  const float c1 = c12.x * inv_n, c2 = c12.y * inv_n;
  for (int i = 0; i < loops; ++i) {
    float d[V], n[V];
    const int64_t off = fetch(i, d, n);
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = rstd * (d[j] - c1 - n[j] * c2);
    char* out = a.out + row * a.outpitch;
    if (ALIGNED && off + 16 <= a.row_bytes) *reinterpret_cast<uint4*>(out + off) = E::pack(d);
    else store_unit<DT, ALIGNED>(out, off, a.row_bytes, E::pack(d));
  }
}

// Column sums of wide rows: block (x, y) adds rows y, y + gridDim.y, ... of
// 256 units into partial row y.
template <int DT, bool CKPT, bool ALIGNED>
__global__ void __launch_bounds__(256) norm_columns_kernel(const __grid_constant__ NormArgs a) {
  constexpr int V = Elem<DT>::V;
  const int64_t off = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 16;
  const int64_t c = off / elem_size(DT);
  float sg[V] = {}, sb[V] = {};
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float d[V], n[V];
    RawUnit<DT, CKPT> r;
    load_raw<DT, CKPT, ALIGNED>(r, a, row, off);
    unpack_raw<DT, CKPT>(r, d, n);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      sg[j] = fmaf(d[j], (n[j] - mean) * rstd, sg[j]);
      sb[j] += d[j];
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (c + j < a.cols) put_sums(a, blockIdx.y, gridDim.y == 1, c + j, sg[j], sb[j]);
}

// out[c] (+)= the sum of part[p][which][c] over p: a block takes 32 columns
// of one of the two sums; its 32 warps add every 32nd partial row in order,
// then the warps' sums are added in warp order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* part, int parts,
                                                          int64_t cols, float* dgamma,
                                                          float* dbeta, int accumulate) {
  __shared__ float s[32][33];
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) {
    after_previous();
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.0f;
  after_previous();
  if (c < cols) {
    const float* p = part + (int64_t)blockIdx.y * cols + c;
    const int64_t pitch = 2 * cols;
#pragma unroll 4
    for (int i = warp; i < parts; i += 32) v += p[i * pitch];
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < cols) {
    v = s[0][lane];
#pragma unroll
    for (int w = 1; w < 32; ++w) v += s[w][lane];
    out[c] = accumulate ? out[c] + v : v;
  }
}

// --- host ----------------------------------------------------------------------------------------

constexpr int kMaxSms = 160;  // the scratch is sized for at most so many

// Rows of 513 .. 16384 columns (8192 backward) go through the ring while two
// stages fit.
struct RingPlan {
  int threads;  // of the rows; 0: not this way
  uint32_t second_at, scales_at, stage_bytes, smem;
  int stages, per_sm, rows;  // rows: of a forward block at once
};

// Dynamic shared memory that each of n blocks of an SM may use: 228 KB less
// the system's 1 KB a block and the kernels' static part (two turns of 2 x 36
// sums, a full and, backward, an empty barrier per stage).
constexpr int64_t kStaticSmem =
    (2 * 36 * 2 * sizeof(float) + 2 * kMaxStages * sizeof(uint64_t) + 127) / 128 * 128;
int64_t block_smem(int n) { return 228 * 1024 / n - 1024 - kStaticSmem; }

// Threads of a row; 0 where rows are too narrow or too wide.  (A wider row's
// threads would leave an SM a single block of more registers: 11008 columns
// ran at 31% of the copy rate backward, against 61% for the passes that read
// a row twice.)
int ring_threads(int64_t cols, bool back) {
  const int64_t c = ckpt_codes_pitch(cols);
  const int threads = back ? 512 : forward_warps(1) * 32;
  return c <= 512 || c > threads * kCols ? 0 : (int)round_up(ceil_div(c, kCols), 32);
}

// Blocks of the backward kernel per SM by registers, the producer warp counted.
int backward_blocks(int threads) { return std::max(1, kBackwardWarps / (threads / 32 + 1)); }

RingPlan ring_plan(int64_t cols, int dtype, bool back, bool ckpt) {
  RingPlan p{};
  p.threads = ring_threads(cols, back);
  if (!p.threads) return p;
  const int64_t c = ckpt_codes_pitch(cols);
  const int64_t row = round_up(cols * elem_size(dtype) + 15, 16) + 16;  // with a shifted start
  p.second_at = (uint32_t)round_up(row, 128);
  int64_t bytes = p.second_at;
  if (back) bytes += ckpt ? c : round_up(row, 128);
  p.scales_at = (uint32_t)round_up(bytes, 128);
  if (back && ckpt) bytes = p.scales_at + ckpt_scales_pitch(cols);
  p.stage_bytes = (uint32_t)round_up(bytes, 128);
  const int64_t params = (int64_t)p.threads * kCols * (back ? 4 : 8);
  // as many blocks as registers allow, fewer where two stages do not fit
  p.rows = forward_rows(c, dtype);
  p.per_sm = back ? backward_blocks(p.threads) : forward_warps(p.rows) / (p.threads / 32);
  while (p.per_sm > 1 && params + 2 * (int64_t)p.stage_bytes > block_smem(p.per_sm)) --p.per_sm;
  p.stages =
      (int)std::min<int64_t>(kMaxStages, (block_smem(p.per_sm) - params) / p.stage_bytes);
  if (p.stages < 2) return RingPlan{};  // two rows at once need two
  p.smem = (uint32_t)(p.stages * (int64_t)p.stage_bytes + params);
  return p;
}

void apply(NormArgs& a, const RingPlan& p, const gc_ctx* ctx) {
  a.status = ctx->ws.status;
  a.second_at = p.second_at;
  a.scales_at = p.scales_at;
  a.stage_bytes = p.stage_bytes;
  a.stages = p.stages;
}

template <auto Kernel>
void launch_ring(gc_ctx* ctx, const NormArgs& a, const RingPlan& p, unsigned grid, int threads) {
  static uint64_t devices = 0;
  if (!allow_smem(ctx, Kernel, (int)block_smem(1), devices)) return;  // the launch's error says so
  Kernel<<<grid, threads, p.smem, ctx->stream>>>(a);
}

template <int DT, int K>
void forward_block(gc_ctx* ctx, const NormArgs& a, int threads, bool aligned) {
  if (aligned)
    norm_forward_kernel<DT, K, true><<<(unsigned)a.rows, threads, 0, ctx->stream>>>(a);
  else
    norm_forward_kernel<DT, K, false><<<(unsigned)a.rows, threads, 0, ctx->stream>>>(a);
}

template <int DT, int K>
void forward_warp(gc_ctx* ctx, const NormArgs& a, bool aligned) {
  const unsigned g = (unsigned)std::min<int64_t>(ceil_div(a.rows, 8),
                                                 (int64_t)ctx->num_sms * 4);
  const size_t smem = (size_t)K * 32 * Elem<DT>::V * 8;
  if (aligned)
    norm_forward_warp_kernel<DT, K, true><<<g, 256, smem, ctx->stream>>>(a);
  else
    norm_forward_warp_kernel<DT, K, false><<<g, 256, smem, ctx->stream>>>(a);
}

template <int DT, int R>
void forward_ring(gc_ctx* ctx, const NormArgs& a, const RingPlan& p, bool aligned) {
  const unsigned g = (unsigned)std::min<int64_t>(a.rows, (int64_t)ctx->num_sms * p.per_sm);
  if (!aligned) launch_ring<norm_forward_ring_kernel<DT, R, kAnywhere>>(ctx, a, p, g, p.threads);
  else if (a.cols == (int64_t)p.threads * kCols)
    launch_ring<norm_forward_ring_kernel<DT, R, kFull>>(ctx, a, p, g, p.threads);
  else launch_ring<norm_forward_ring_kernel<DT, R, kEnds>>(ctx, a, p, g, p.threads);
}

template <int DT>
void forward_dt(gc_ctx* ctx, NormArgs& a, bool aligned) {
  const int64_t units = a.codes_pitch / Elem<DT>::V;
  // fewer rows than SMs: a block each, one unit per thread
  if (units > 32 && units <= 1024 && a.rows <= ctx->num_sms) {
    forward_block<DT, 1>(ctx, a, (int)round_up(units, 32), aligned);
  } else if (a.codes_pitch <= 512) {
    if (units <= 32) forward_warp<DT, 1>(ctx, a, aligned);
    else if (DT != GC_F32 || units <= 64) forward_warp<DT, 2>(ctx, a, aligned);
    else forward_warp<DT, DT == GC_F32 ? 4 : 2>(ctx, a, aligned);  // fp32: 4 columns a unit
  } else {
    const RingPlan p = ring_plan(a.cols, DT, false, false);
    if (p.threads) {
      apply(a, p, ctx);
      if (DT != GC_F32 && p.rows == 2) forward_ring<DT, DT == GC_F32 ? 1 : 2>(ctx, a, p, aligned);
      else forward_ring<DT, 1>(ctx, a, p, aligned);
    } else {
      forward_block<DT, 0>(ctx, a, 1024, aligned);
    }
  }
}

// Partial rows of the column sums that a call may leave.
int64_t max_parts(int64_t cols) {
  const int threads = ring_threads(cols, true);
  return (int64_t)kMaxSms * (threads ? backward_blocks(threads) : 2);
}

template <int DT, bool CKPT>
int backward_ring(gc_ctx* ctx, const NormArgs& a, const RingPlan& p, bool aligned) {
  const unsigned g =
      (unsigned)std::min<int64_t>(a.rows, (int64_t)std::min(ctx->num_sms, kMaxSms) * p.per_sm);
  const int threads = p.threads + 32;
  if (!aligned) launch_ring<norm_backward_ring_kernel<DT, CKPT, kAnywhere>>(ctx, a, p, g, threads);
  else if (a.cols == (int64_t)p.threads * kCols)
    launch_ring<norm_backward_ring_kernel<DT, CKPT, kFull>>(ctx, a, p, g, threads);
  else launch_ring<norm_backward_ring_kernel<DT, CKPT, kEnds>>(ctx, a, p, g, threads);
  return (int)g;
}

template <int DT, int K, bool CKPT>
void backward_launch(gc_ctx* ctx, const NormArgs& a, unsigned grid, bool aligned) {
  const size_t smem = (size_t)a.codes_pitch * 2 * sizeof(float);
  if (aligned)
    norm_backward_kernel<DT, K, CKPT, true><<<grid, 256, smem, ctx->stream>>>(a);
  else
    norm_backward_kernel<DT, K, CKPT, false><<<grid, 256, smem, ctx->stream>>>(a);
}

// Launches the row pass; returns the partial rows of the column sums.
template <int DT, bool CKPT>
int backward_dt(gc_ctx* ctx, NormArgs& a, bool aligned) {
  constexpr int V = Elem<DT>::V;
  const int64_t sms = std::min(ctx->num_sms, kMaxSms);
  if (a.codes_pitch <= 512) {
    LaunchScope L(ctx, GC_PHASE_NORM_BACKWARD);
    const unsigned g = (unsigned)std::min<int64_t>(ceil_div(a.rows, 8), sms * 2);
    backward_launch<DT, 16 / V, CKPT>(ctx, a, g, aligned);
    return (int)g;
  }
  const RingPlan p = ring_plan(a.cols, DT, true, CKPT);
  if (p.threads) {
    LaunchScope L(ctx, GC_PHASE_NORM_BACKWARD);
    apply(a, p, ctx);
    return backward_ring<DT, CKPT>(ctx, a, p, aligned);
  }
  {
    LaunchScope L(ctx, GC_PHASE_NORM_BACKWARD);
    if (aligned)
      norm_backward_wide_kernel<DT, CKPT, true><<<(unsigned)a.rows, 512, 0, ctx->stream>>>(a);
    else
      norm_backward_wide_kernel<DT, CKPT, false><<<(unsigned)a.rows, 512, 0, ctx->stream>>>(a);
  }
  if (!a.dgamma && !a.dbeta) return 0;
  LaunchScope L(ctx, GC_PHASE_NORM_BACKWARD);
  const int64_t bx = ceil_div(a.codes_pitch / V, 256);
  const int64_t by = std::max<int64_t>(
      1, std::min<int64_t>({ceil_div(a.rows, 16), sms * 2, ceil_div(sms * 8, bx)}));
  const dim3 g((unsigned)bx, (unsigned)by);
  if (aligned)
    norm_columns_kernel<DT, CKPT, true><<<g, 256, 0, ctx->stream>>>(a);
  else
    norm_columns_kernel<DT, CKPT, false><<<g, 256, 0, ctx->stream>>>(a);
  return (int)by;
}

template <int DT>
gc_status backward_all(gc_ctx* ctx, NormArgs& a, bool aligned) {
  int parts = 0;
  if (a.rows > 0)
    parts = a.codes ? backward_dt<DT, true>(ctx, a, aligned) : backward_dt<DT, false>(ctx, a, aligned);
  if ((a.dgamma || a.dbeta) && parts != 1) {
    LaunchScope L(ctx, GC_PHASE_NORM_REDUCE);
    if (launch_early(norm_reduce_kernel, dim3((unsigned)ceil_div(a.cols, 32), 2), 1024, 0,
                     ctx->stream, a.part, parts, a.cols, a.dgamma, a.dbeta,
                     a.accumulate) != cudaSuccess)
      return GC_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

const char* end_of(const void* p, int64_t ld, int dtype, int64_t rows, int64_t cols) {
  return static_cast<const char*>(p) + ((rows - 1) * ld + cols) * elem_size(dtype);
}

}  // namespace

int64_t norm_scratch_bytes(int64_t rows, int64_t cols) {
  const int64_t parts = std::min<int64_t>(rows, max_parts(cols));
  return parts * 2 * cols * (int64_t)sizeof(float);
}

gc_status launch_norm_forward(gc_ctx* ctx, const void* x, int dtype, int64_t rows, int64_t cols,
                              int64_t ldx, const void* gamma, const void* beta, int ptype,
                              float eps, void* y, int64_t ldy, float* mean, float* rstd,
                              uint8_t* codes, uint8_t* scales) {
  if (rows == 0 || cols == 0) return GC_OK;
  const int e = elem_size(dtype);
  NormArgs a{};
  a.x = static_cast<const char*>(x);
  a.xend = end_of(x, ldx, dtype, rows, cols);
  a.out = static_cast<char*>(y);
  a.gamma = gamma;
  a.beta = beta;
  a.mean = mean;
  a.rstd = rstd;
  a.codes = codes;
  a.scales = scales;
  a.rows = rows;
  a.cols = cols;
  a.row_bytes = cols * e;
  a.xpitch = ldx * e;
  a.outpitch = ldy * e;
  a.codes_pitch = ckpt_codes_pitch(cols);
  a.scales_pitch = ckpt_scales_pitch(cols);
  a.eps = eps;
  a.ptype = ptype;
  const bool aligned = row_aligned(ldx, dtype) && row_aligned(ldy, dtype);
  LaunchScope L(ctx, GC_PHASE_NORM_FORWARD);
  if (dtype == GC_F32) forward_dt<GC_F32>(ctx, a, aligned);
  else if (dtype == GC_BF16) forward_dt<GC_BF16>(ctx, a, aligned);
  else forward_dt<GC_F16>(ctx, a, aligned);
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

gc_status launch_norm_backward(gc_ctx* ctx, const void* dy, int64_t lddy, const void* x,
                               int64_t ldx, const uint8_t* codes, const uint8_t* scales, int dtype,
                               int64_t rows, int64_t cols, const void* gamma, int ptype,
                               const float* mean, const float* rstd, void* dx, int64_t lddx,
                               float* dgamma, float* dbeta, int accumulate, float* part) {
  if (cols == 0) return GC_OK;
  const int e = elem_size(dtype);
  NormArgs a{};
  a.x = static_cast<const char*>(x);
  a.dy = static_cast<const char*>(dy);
  if (x) a.xend = end_of(x, ldx, dtype, rows, cols);
  a.dyend = end_of(dy, lddy, dtype, rows, cols);
  a.out = static_cast<char*>(dx);
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
  a.row_bytes = cols * e;
  a.xpitch = ldx * e;
  a.dypitch = lddy * e;
  a.outpitch = lddx * e;
  a.codes_pitch = ckpt_codes_pitch(cols);
  a.scales_pitch = ckpt_scales_pitch(cols);
  a.ptype = ptype;
  a.accumulate = accumulate;
  const bool aligned = row_aligned(lddy, dtype) && row_aligned(lddx, dtype) &&
                       (codes || row_aligned(ldx, dtype));
  if (dtype == GC_F32) return backward_all<GC_F32>(ctx, a, aligned);
  if (dtype == GC_BF16) return backward_all<GC_BF16>(ctx, a, aligned);
  return backward_all<GC_F16>(ctx, a, aligned);
}

}  // namespace gc
