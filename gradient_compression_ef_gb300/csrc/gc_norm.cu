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
//   cols <= 1024        a warp per row, up to 4 units of 16 bytes per lane;
//   wider, while two    a block walks over rows that one thread copies into a
//   rows fit in shared  ring of stages in shared memory (bulk copies, several
//   memory              rows ahead); a thread owns 16 or 32 columns for all
//                       rows: parameters and column sums stay in registers,
//                       and nothing but the stage changes from row to row;
//   wider still         the row is read again from L2 for each of its passes.
// The backward pass leaves one partial row of column sums per block; a second
// small grid adds the partials in block order.
#include <algorithm>

#include "gc_act8.cuh"
#include "gc_sm100.cuh"

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

// K units per thread, unit i of a thread being thread + i * threads.  K == 0:
// rows wider than the registers hold; the row is read again (from L2) for
// each of its three passes.
template <int DT, int K, bool WARP, bool ALIGNED>
__global__ void __launch_bounds__(WARP ? 256 : 1024)
    norm_forward_kernel(const __grid_constant__ NormArgs a) {
  using E = Elem<DT>;
  constexpr int V = E::V, KK = K ? K : 1;
  __shared__ float2 slot[2][32];
  RowSum<WARP> sum{slot};
  const int nt = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5)
                           : (int64_t)blockIdx.x;
  if (row >= a.rows) return;  // whole warps only, no barrier follows for WARP
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
  r.dy = load_unit<DT, ALIGNED>(a.dy + row * a.dypitch, off, a.row_bytes, a.dyend);
  if constexpr (CKPT) {
    const int64_t c = off / elem_size(DT);
    r.c = Codes<V>{};
    r.b = 0u;
    if (c < a.codes_pitch) {
      r.c = load_codes<V>(a.codes + row * a.codes_pitch + c);
      r.b = __ldg(a.scales + row * a.scales_pitch + c / kActGroup);
    }
  } else {
    r.x = load_unit<DT, ALIGNED>(a.x + row * a.xpitch, off, a.row_bytes, a.xend);
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
  float* pg = a.part + (int64_t)blockIdx.x * 2 * a.cols;
  float* pb = pg + a.cols;
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
  for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
    pg[c] = acc[c];
    pb[c] = acc[w8 + c];
  }
}

// ---------------------------------------------------------------------------
// Rows through a ring of stages in shared memory.
// ---------------------------------------------------------------------------
constexpr int kMaxStages = 4;
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

__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds_u128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// A unit from a staged row whose first byte lies `mis` bytes into it; `left`
// of the row's bytes begin at the unit (the columns past them are zero).
template <int DT, bool ALIGNED>
__device__ __forceinline__ uint4 staged_unit(uint32_t at, uint32_t mis, int left) {
  uint4 r;
  if (ALIGNED) {
    r = lds_u128(at);
  } else {
    const uint32_t p = at + (mis & ~3u);
    uint32_t w[5];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = lds_u32(p + 4 * i);
    if (elem_size(DT) == 2 && (mis & 2u)) {
      w[4] = lds_u32(p + 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (left < 16) {
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

// Block-wide sums for the ring kernels; the barrier also carries whether a
// thread's wait ran out (then every thread leaves its row loop).
struct BlockSum {
  float2 (*slot)[32];
  int turn = 0;
  __device__ __forceinline__ float2 operator()(float a, float b, bool& ok) {
    a = warp_allsum(a);
    b = warp_allsum(b);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0) slot[turn][warp] = make_float2(a, b);
    ok = !__syncthreads_or(!ok);
    const float2 v = lane < nw ? slot[turn][lane] : make_float2(0.0f, 0.0f);
    turn ^= 1;
    return make_float2(warp_allsum(v.x), warp_allsum(v.y));
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

// E columns per thread, unit i of a thread being thread + i * threads.
template <int DT, int E, bool ALIGNED>
__global__ void __launch_bounds__(512, 1)
    norm_forward_ring_kernel(const __grid_constant__ NormArgs a) {
  using namespace sm100;
  using L = Elem<DT>;
  constexpr int V = L::V, K = E / V;
  extern __shared__ __align__(128) char stages[];
  __shared__ float2 slot[2][32];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  BlockSum sum{slot};
  const int t = threadIdx.x, nt = blockDim.x;
  if (t == 0) {
    for (int i = 0; i < a.stages; ++i) mbar_init(&full[i], 1);
    mbar_fence_init();
    int64_t r = blockIdx.x;
    for (int i = 0; i < a.stages && r < a.rows; ++i, r += gridDim.x)
      fill_stage<DT, false, false>(a, r, stages + i * a.stage_bytes, &full[i]);
  }
  const uint32_t base = smem_u32(stages);
  const float inv_n = 1.0f / (float)a.cols;
  float g[K][V], b[K][V];
  int left[K];  // bytes of the row from the unit on
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int64_t u = t + (int64_t)i * nt;
    left[i] = (int)max((int64_t)0, min((int64_t)16, a.row_bytes - u * 16));
    load_params<V>(g[i], a.gamma, a.ptype, u * V, a.cols, 1.0f);
    load_params<V>(b[i], a.beta, a.ptype, u * V, a.cols, 0.0f);
  }
  __syncthreads();
  bool ok = true;
  RingPos ring;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ring.next(a.stages)) {
    ok = mbar_wait(&full[ring.st], ring.ph, kWaitCycles);
    const uint32_t stage = base + ring.st * a.stage_bytes;
    const uint32_t mis =
        ALIGNED ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(a.x + row * a.xpitch) & 15u);
    uint4 raw[K];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      raw[i] = left[i] > 0 ? staged_unit<DT, ALIGNED>(stage + (t + i * nt) * 16, mis, left[i])
                           : make_uint4(0u, 0u, 0u, 0u);
      float v[V];
      L::unpack(raw[i], v);
#pragma unroll
      for (int j = 0; j < V; ++j) s += v[j];
    }
    const float mean = sum(s, 0.0f, ok).x * inv_n;
    if (!ok) break;
    // every thread holds its part of the row: the stage takes a later one
    if (t == 0 && row + (int64_t)a.stages * gridDim.x < a.rows) {
      fence_proxy_async_smem();
      fill_stage<DT, false, false>(a, row + (int64_t)a.stages * gridDim.x,
                                   stages + ring.st * a.stage_bytes, &full[ring.st]);
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      keep_packed(raw[i]);
      float v[V];
      L::unpack(raw[i], v);
      if (left[i] == 16) {
#pragma unroll
        for (int j = 0; j < V; ++j) q = fmaf(v[j] - mean, v[j] - mean, q);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (j * elem_size(DT) < left[i]) q = fmaf(v[j] - mean, v[j] - mean, q);
      }
    }
    const float rstd = rsqrtf(sum(q, 0.0f, ok).x * inv_n + a.eps);
    if (t == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    char* out = a.out + row * a.outpitch;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      keep_packed(raw[i]);
      float v[V];
      L::unpack(raw[i], v);
      const uint32_t u = t + i * nt;
      if (a.codes) {
        const uint32_t sb = scale_byte(group_max_bits<DT>(raw[i]));
        if (u * V < a.codes_pitch) {
          store_codes<DT>(a.codes + row * a.codes_pitch + u * V, raw[i], v, sb);
          if (t % (kActGroup / V) == 0)
            a.scales[row * a.scales_pitch + u * V / kActGroup] = (uint8_t)sb;
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = fmaf((v[j] - mean) * rstd, g[i][j], b[i][j]);
      const uint4 r = L::pack(v);
      if (ALIGNED && left[i] == 16) *reinterpret_cast<uint4*>(out + u * 16) = r;
      else store_unit<DT, ALIGNED>(out, (int64_t)u * 16, a.row_bytes, r);
    }
  }
  ring_end(ok, a.status);
}

// E columns per thread.  With 16 a thread keeps d and n between the two
// passes over the row, and gamma; with 32 it takes them from the stage and
// from L1 again (the column sums alone are 64 registers).
template <int DT, int E, bool CKPT, bool ALIGNED>
__global__ void __launch_bounds__(512, 1)
    norm_backward_ring_kernel(const __grid_constant__ NormArgs a) {
  using namespace sm100;
  using L = Elem<DT>;
  constexpr int V = L::V, K = E / V;
  constexpr bool KEEP = E == 16;
  extern __shared__ __align__(128) char stages[];
  __shared__ float2 slot[2][32];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  BlockSum sum{slot};
  const int t = threadIdx.x, nt = blockDim.x;
  int64_t fetch = blockIdx.x;  // next row to copy (thread 0)
  if (t == 0) {
    for (int i = 0; i < a.stages; ++i) mbar_init(&full[i], 1);
    mbar_fence_init();
    for (int i = 0; i < a.stages && fetch < a.rows; ++i, fetch += gridDim.x)
      fill_stage<DT, true, CKPT>(a, fetch, stages + i * a.stage_bytes, &full[i]);
  }
  const uint32_t base = smem_u32(stages);
  const float inv_n = 1.0f / (float)a.cols;
  float sg[K][V], sb[K][V], gk[KEEP ? K : 1][V];
  int left[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int64_t u = t + (int64_t)i * nt;
    left[i] = (int)max((int64_t)0, min((int64_t)16, a.row_bytes - u * 16));
    if (KEEP) load_params<V>(gk[KEEP ? i : 0], a.gamma, a.ptype, u * V, a.cols, 1.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) sg[i][j] = sb[i][j] = 0.0f;
  }
  float mean_n = 0.0f, rstd_n = 0.0f;
  if (blockIdx.x < a.rows) {
    mean_n = __ldg(a.mean + blockIdx.x);
    rstd_n = __ldg(a.rstd + blockIdx.x);
  }
  __syncthreads();
  bool ok = true;
  RingPos ring;
  int last_st = -1;  // the stage of the row before
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ring.next(a.stages)) {
    ok = mbar_wait(&full[ring.st], ring.ph, kWaitCycles);
    const uint32_t stage = base + ring.st * a.stage_bytes;
    const float mean = mean_n, rstd = rstd_n;
    if (row + gridDim.x < a.rows) {
      mean_n = __ldg(a.mean + row + gridDim.x);
      rstd_n = __ldg(a.rstd + row + gridDim.x);
    }
    const uint32_t mis0 =
        ALIGNED ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(a.dy + row * a.dypitch) & 15u);
    const uint32_t mis1 =
        ALIGNED ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(a.x + row * a.xpitch) & 15u);
    // dy and n = (x - mean) rstd of unit i
    auto inputs = [&](int i, float (&d)[V], float (&n)[V]) {
      const uint32_t u = t + i * nt;
      L::unpack(staged_unit<DT, ALIGNED>(stage + u * 16, mis0, left[i]), d);
      if (CKPT) {
        Codes<V> c;
#pragma unroll
        for (int w = 0; w < V / 4; ++w) c.w[w] = lds_u32(stage + a.second_at + u * V + 4 * w);
        uint32_t bb;
        asm volatile("ld.shared.u8 %0, [%1];"
                     : "=r"(bb)
                     : "r"(stage + a.scales_at + u * V / kActGroup)
                     : "memory");
        decode<V>(n, c, bb);
      } else {
        L::unpack(staged_unit<DT, ALIGNED>(stage + a.second_at + u * 16, mis1, left[i]), n);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) n[j] = (n[j] - mean) * rstd;
    };
    auto gamma = [&](int i, float (&g)[V]) {
      if (KEEP) {
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] = gk[KEEP ? i : 0][j];
      } else {
        load_params<V>(g, a.gamma, a.ptype, ((int64_t)t + (int64_t)i * nt) * V, a.cols, 1.0f);
      }
    };
    float dk[KEEP ? K : 1][V], nk[KEEP ? K : 1][V];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float (&d)[V] = dk[KEEP ? i : 0];
      float (&n)[V] = nk[KEEP ? i : 0];
      if (left[i] > 0) {
        float g[V];
        inputs(i, d, n);
        gamma(i, g);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          sg[i][j] = fmaf(d[j], n[j], sg[i][j]);
          sb[i][j] += d[j];
          d[j] *= g[j];  // dy is 0 past the last column
          s1 += d[j];
          s2 = fmaf(d[j], n[j], s2);
        }
      }
    }
    const float2 c12 = sum(s1, s2, ok);
    if (!ok) break;
    // all threads are past the row before: its stage takes the next row
    if (t == 0) {
      if (last_st >= 0 && fetch < a.rows) {
        fence_proxy_async_smem();
        fill_stage<DT, true, CKPT>(a, fetch, stages + last_st * a.stage_bytes, &full[last_st]);
        fetch += gridDim.x;
      }
      last_st = ring.st;
    }
    const float c1 = c12.x * inv_n * rstd, c2 = c12.y * inv_n * rstd;
    char* out = a.out + row * a.outpitch;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const uint32_t u = t + i * nt;
      float o[V];
      if (KEEP) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          o[j] = fmaf(rstd, dk[KEEP ? i : 0][j], fmaf(-c2, nk[KEEP ? i : 0][j], -c1));
      } else {
        float n[V], g[V];
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = 0.0f;
        if (left[i] > 0) {
          inputs(i, o, n);
          gamma(i, g);
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] = fmaf(rstd, o[j] * g[j], fmaf(-c2, n[j], -c1));
        }
      }
      const uint4 r = L::pack(o);
      if (ALIGNED && left[i] == 16) *reinterpret_cast<uint4*>(out + u * 16) = r;
      else store_unit<DT, ALIGNED>(out, (int64_t)u * 16, a.row_bytes, r);
    }
  }
  ring_end(ok, a.status);

  if (!a.dgamma && !a.dbeta) return;
  float* pg = a.part + (int64_t)blockIdx.x * 2 * a.cols;
  float* pb = pg + a.cols;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int64_t c = ((int64_t)t + (int64_t)i * nt) * V;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (c + j < a.cols) {
        pg[c + j] = sg[i][j];
        pb[c + j] = sb[i][j];
      }
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
    store_unit<DT, ALIGNED>(a.out + row * a.outpitch, off, a.row_bytes, E::pack(d));
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
  float* pg = a.part + (int64_t)blockIdx.y * 2 * a.cols;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (c + j < a.cols) {
      pg[c + j] = sg[j];
      pg[a.cols + c + j] = sb[j];
    }
}

// out[c] (+)= the sum of part[p][which][c] over p: a block takes 32 columns
// of one of the two sums; its 16 warps add every 16th partial row in order,
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
  if (c < cols) {
    const float* p = part + (int64_t)blockIdx.y * cols + c;
    const int64_t pitch = 2 * cols;
#pragma unroll 4
    for (int i = warp; i < parts; i += 16) v += p[i * pitch];
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < cols) {
    v = s[0][lane];
#pragma unroll
    for (int w = 1; w < 16; ++w) v += s[w][lane];
    out[c] = accumulate ? out[c] + v : v;
  }
}

// --- host ----------------------------------------------------------------------------------------

constexpr int kMaxSms = 160;  // the scratch is sized for at most so many

// Rows of 1025 .. 16384 columns go through the ring while two stages fit;
// E columns per thread.
struct RingPlan {
  int e, threads;  // e == 0: not this way
  uint32_t second_at, scales_at, stage_bytes;
  int stages, per_sm;
};

constexpr uint32_t kRingBytes = 216 * 1024;  // of an SM's shared memory

RingPlan ring_plan(int64_t cols, int dtype, bool back, bool ckpt) {
  RingPlan p{};
  const int64_t c = ckpt_codes_pitch(cols);
  if (c <= 1024 || c > 512 * 32) return p;
  const int64_t row = round_up(cols * elem_size(dtype) + 15, 16) + 16;  // with a shifted start
  p.second_at = (uint32_t)round_up(row, 128);
  int64_t bytes = p.second_at;
  if (back) bytes += ckpt ? c : round_up(row, 128);
  p.scales_at = (uint32_t)round_up(bytes, 128);
  if (back && ckpt) bytes = p.scales_at + ckpt_scales_pitch(cols);
  p.stage_bytes = (uint32_t)round_up(bytes, 128);
  if (2 * p.stage_bytes > kRingBytes) return p;
  p.e = c <= 512 * 16 ? 16 : 32;
  p.threads = (int)round_up(ceil_div(c, p.e), 32);
  // blocks per SM by registers (128 a thread), then as many stages as fit
  p.per_sm = std::max(1, 512 / p.threads);
  while (p.per_sm > 1 && 2 * p.stage_bytes > kRingBytes / p.per_sm) --p.per_sm;
  p.stages = (int)std::min<int64_t>(kMaxStages, kRingBytes / p.per_sm / p.stage_bytes);
  return p;
}

void apply(NormArgs& a, const RingPlan& p, const gc_ctx* ctx) {
  a.status = ctx->ws.status;
  a.second_at = p.second_at;
  a.scales_at = p.scales_at;
  a.stage_bytes = p.stage_bytes;
  a.stages = p.stages;
}

template <class Kernel>
void launch_ring(Kernel kernel, gc_ctx* ctx, const NormArgs& a, const RingPlan& p, unsigned grid) {
  const int smem = (int)(p.stage_bytes * p.stages);
  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  kernel<<<grid, p.threads, smem, ctx->stream>>>(a);
}

template <int DT, int K, bool WARP>
void forward_launch(gc_ctx* ctx, const NormArgs& a, int threads, bool aligned) {
  const int per_block = WARP ? threads / 32 : 1;
  const unsigned grid = (unsigned)ceil_div(a.rows, per_block);
  if (aligned)
    norm_forward_kernel<DT, K, WARP, true><<<grid, threads, 0, ctx->stream>>>(a);
  else
    norm_forward_kernel<DT, K, WARP, false><<<grid, threads, 0, ctx->stream>>>(a);
}

template <int DT>
void forward_dt(gc_ctx* ctx, NormArgs& a, bool aligned) {
  const int64_t units = a.codes_pitch / Elem<DT>::V;
  const RingPlan p = ring_plan(a.cols, DT, false, false);
  // fewer rows than SMs: a block each, one unit per thread
  if (units <= 1024 && units > 32 && a.rows <= ctx->num_sms) {
    forward_launch<DT, 1, false>(ctx, a, (int)round_up(units, 32), aligned);
  } else if (p.e) {
    apply(a, p, ctx);
    const unsigned g = (unsigned)std::min<int64_t>(a.rows, (int64_t)ctx->num_sms * p.per_sm);
    if (p.e == 16) {
      if (aligned) launch_ring(norm_forward_ring_kernel<DT, 16, true>, ctx, a, p, g);
      else launch_ring(norm_forward_ring_kernel<DT, 16, false>, ctx, a, p, g);
    } else {
      if (aligned) launch_ring(norm_forward_ring_kernel<DT, 32, true>, ctx, a, p, g);
      else launch_ring(norm_forward_ring_kernel<DT, 32, false>, ctx, a, p, g);
    }
  } else if (units <= 32) {
    forward_launch<DT, 1, true>(ctx, a, 256, aligned);
  } else if (units <= 64) {
    forward_launch<DT, 2, true>(ctx, a, 256, aligned);
  } else if (units <= 128) {
    forward_launch<DT, 4, true>(ctx, a, 256, aligned);
  } else if (units <= 256) {  // fp32, 513 .. 1024 columns
    forward_launch<DT, 8, true>(ctx, a, 256, aligned);
  } else {
    forward_launch<DT, 0, false>(ctx, a, 1024, aligned);
  }
}

// Partial rows of the column sums that a call may leave.
int64_t max_parts(int64_t cols) {
  const int64_t c = ckpt_codes_pitch(cols);
  if (c <= 1024) return kMaxSms * 2;
  const int threads = (int)round_up(ceil_div(c, c <= 512 * 16 ? 16 : 32), 32);
  return (int64_t)kMaxSms * std::max(2, 512 / threads);
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
  if (a.codes_pitch <= 1024) {
    LaunchScope L(ctx, GC_PHASE_NORM_BACKWARD);
    const unsigned g = (unsigned)std::min<int64_t>(ceil_div(a.rows, 8), sms * 2);
    if (a.codes_pitch <= 512) backward_launch<DT, 16 / V, CKPT>(ctx, a, g, aligned);
    else backward_launch<DT, 32 / V, CKPT>(ctx, a, g, aligned);
    return (int)g;
  }
  const RingPlan p = ring_plan(a.cols, DT, true, CKPT);
  if (p.e) {
    LaunchScope L(ctx, GC_PHASE_NORM_BACKWARD);
    apply(a, p, ctx);
    const unsigned g = (unsigned)std::min<int64_t>(a.rows, sms * p.per_sm);
    if (p.e == 16) {
      if (aligned) launch_ring(norm_backward_ring_kernel<DT, 16, CKPT, true>, ctx, a, p, g);
      else launch_ring(norm_backward_ring_kernel<DT, 16, CKPT, false>, ctx, a, p, g);
    } else {
      if (aligned) launch_ring(norm_backward_ring_kernel<DT, 32, CKPT, true>, ctx, a, p, g);
      else launch_ring(norm_backward_ring_kernel<DT, 32, CKPT, false>, ctx, a, p, g);
    }
    return (int)g;
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
  if (a.dgamma || a.dbeta) {
    LaunchScope L(ctx, GC_PHASE_NORM_REDUCE);
    norm_reduce_kernel<<<dim3((unsigned)ceil_div(a.cols, 32), 2), 512, 0, ctx->stream>>>(
        a.part, parts, a.cols, a.dgamma, a.dbeta, a.accumulate);
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
