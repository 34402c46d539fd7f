// gc_embed.cu -- embedding lookup with a scale, and the table's gradient.
//
//   forward   y[t] = scale table[ids[t]]            (pad: zeros)
//   gradient  dtable[v] (+)= scale sum of dy[t] over the tokens t with
//             ids[t] = v, in ascending order of t
//
// Up to 256 tokens take one launch: the first token of each id sums the rows of
// all that have it.  More are sorted as (id, token) pairs, stable, and runs of
// one id are summed:
//   sort      up to 8192 tokens: each pair's place is the number of pairs
//             before it, counted (1000, 2500, 5003, 8192 tokens, each launch
//             timed by events: 7, 8, 15, 21 us; two radix passes 23 to 24);
//             more: radix passes of up to 9 bits, each of which makes the next
//             one's counts on its way (16384 tokens 18 us)
//   sum       a warp takes 8 to 64 sorted tokens and 512 bytes of their rows,
//             and stores each run's sum once: to the table's row where the run
//             lies inside its tokens, else to a partial row; blocks of their own
//             write zeros to the rows of ids that do not occur
//   join      the partial rows of a run that crosses chunks, in their order
// The order of additions is one that ids and sizes alone decide.
//
// Measured (plain copy: 6.79 TB/s): 16384 tokens, table of 32768 x 4096 bf16:
// lookup 28 us (5.9 TB/s; a table in another type, fp32 to bf16 or back, 72 to 76,
// 4.8 to 4.9), sort 18, sums and zeros 107 (6.2 TB/s), join 8;
// together 167 (floor 126).  5003 x 1001 fp32 on 4-byte boundaries, added to
// 50021 rows: 11 + 13 + 24 + 7 us, launches and round trips, not bytes (floor
// 10).  100 tokens x 512: 3.9 + 6.1 us, of which fetching code is a third.
#include <algorithm>
#include <type_traits>

#include "gc_act8.cuh"

namespace gc {
namespace {

constexpr int kMaxChunk = 64;    // sorted tokens of one unit of work, at most
constexpr int kFew = 256;        // tokens that are not sorted
constexpr int kCountMax = 8192;  // tokens that are sorted by counting
constexpr int kSortBlocks = 128; // blocks of a radix pass, at most
constexpr int kBins = 512;       // digits of up to 9 bits

struct EmbedArgs {
  const void* ids;
  const char *table, *tend;  // forward: the table; gradient: dy
  char* y;
  float *dtable, *part;          // part: [chunks][2][part_pitch]
  uint32_t *key, *tok;           // sorted; key == vocab: no row
  uint32_t* status;
  int64_t tokens, vocab, cols, pad;
  int64_t tpitch, ypitch, ldd, part_pitch;  // bytes, bytes, floats, floats
  int64_t row_bytes;                        // of a row of the table, or of dy
  int64_t zero_blocks;
  float scale;
  int wide_ids, accumulate, chunk;
};

// Radix passes over (key, token) pairs; block b of a pass has the pairs from b
// * tile on.
struct SortArgs {
  const uint32_t *key, *tok;  // NULL: the ids as they come
  uint32_t *key_out, *tok_out;
  uint32_t* count;            // [passes][kCounts]: of this pass, then of those behind it
  int shift, bits, blocks, tile, more;  // more: passes behind this one
};
constexpr int kCounts = kSortBlocks * kBins;

__device__ __forceinline__ int64_t id_at(const void* ids, int wide, int64_t t) {
  return wide ? __ldg(static_cast<const long long*>(ids) + t)
              : (int64_t)__ldg(static_cast<const int*>(ids) + t);
}

// The table's row of token t; -1 for padding and, with the status set, for an
// id outside the table.
__device__ __forceinline__ int64_t row_of(const EmbedArgs& a, int64_t t) {
  const int64_t id = id_at(a.ids, a.wide_ids, t);
  if (id == a.pad) return -1;
  if (id >= 0 && id < a.vocab) return id;
  atomicOr(a.status, kStatusTokenId);
  return -1;
}

// --- forward -------------------------------------------------------------------------------------

template <int DT>
__device__ __forceinline__ uint4 scale_unit(const uint4& r, float s) {
  constexpr int H = Elem<DT>::V / 2;
  float2 v[H];
  unpack2<DT>(r, v);
#pragma unroll
  for (int j = 0; j < H; ++j) v[j] = __fmul2_rn(v[j], both(s));
  return pack2<DT>(v);
}

// One type on both sides: a warp copies runs of U * 512 bytes of a token's row.
template <int DT, int U, bool ALIGNED>
__global__ void __launch_bounds__(256) embed_forward_kernel(const __grid_constant__ EmbedArgs a) {
  const uint32_t segs = (uint32_t)ceil_div(a.row_bytes, (int64_t)(512 * U));
  const int64_t total = a.tokens * segs, step = (int64_t)gridDim.x * 8;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < total; w += step) {
    const int64_t t = w / segs;
    const uint32_t at = (uint32_t)(w - t * segs) * (512u * U);
    const bool inner = (int64_t)at + 512 * U + (ALIGNED ? 0 : 16) <= a.row_bytes;
    const int64_t row = row_of(a, t);
    uint4 r[U];
    if (row >= 0) {
      load_run<DT, ALIGNED>(r, a.table + row * a.tpitch, at, inner, a.row_bytes, a.tend);
#pragma unroll
      for (int i = 0; i < U; ++i) r[i] = scale_unit<DT>(r[i], a.scale);
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) r[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    store_run<DT, ALIGNED>(a.y + t * a.ypitch, at, inner, a.row_bytes, r);
  }
}

template <class T>
__device__ __forceinline__ float to_f32(T v) {
  return (float)v;
}
template <class T>
__device__ __forceinline__ T from_f32(float v) {
  return (T)v;
}
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32(__half v) {
  return __half2float(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32(float v) {
  return __float2half_rn(v);
}

// Two types: four elements per lane, as vectors where rows are aligned.
template <class P, class T, bool ALIGNED>
__global__ void __launch_bounds__(256) embed_cast_kernel(const __grid_constant__ EmbedArgs a) {
  struct alignas(4 * sizeof(P)) P4 { P v[4]; };
  struct alignas(4 * sizeof(T)) T4 { T v[4]; };
  const uint32_t segs = (uint32_t)ceil_div(a.cols, (int64_t)128);
  const int64_t total = a.tokens * segs, step = (int64_t)gridDim.x * 8;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < total; w += step) {
    const int64_t t = w / segs, row = row_of(a, t);
    const int64_t c0 = (w - t * segs) * 128;
    const P* src = reinterpret_cast<const P*>(a.table + (row < 0 ? 0 : row) * a.tpitch);
    T* dst = reinterpret_cast<T*>(a.y + t * a.ypitch);
    const int lane = threadIdx.x & 31;
    if (ALIGNED && c0 + 128 <= a.cols) {
      const int64_t c = c0 + lane * 4;
      P4 p{};
      if (row >= 0) p = *reinterpret_cast<const P4*>(src + c);
      T4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o.v[j] = from_f32<T>(row < 0 ? 0.0f : __fmul_rn(to_f32(p.v[j]), a.scale));
      *reinterpret_cast<T4*>(dst + c) = o;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t c = c0 + j * 32 + lane;
        if (c < a.cols)
          dst[c] = from_f32<T>(row < 0 ? 0.0f : __fmul_rn(to_f32(src[c]), a.scale));
      }
    }
  }
}

// --- sort ----------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t key_of(const EmbedArgs& a, int64_t t) {
  const int64_t row = row_of(a, t);
  return row < 0 ? (uint32_t)a.vocab : (uint32_t)row;
}

// A block places 32 tokens: warp w counts, for the 32 tokens (one per lane),
// the pairs of its share of all tokens that come before.
__global__ void __launch_bounds__(1024) embed_count_kernel(const __grid_constant__ EmbedArgs a) {
  extern __shared__ __align__(16) uint32_t keys[];  // all keys
  const int n = (int)a.tokens, padded = (int)round_up(n, 128);
  __shared__ uint32_t before[32][33];
  let_next_begin();
  for (int t = threadIdx.x; t < padded; t += 1024)
    keys[t] = t < n ? key_of(a, t) : 0xFFFFFFFFu;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int me = blockIdx.x * 32 + lane;
  const uint32_t key = me < n ? keys[me] : 0u;
  uint32_t count = 0;
  for (int j = warp * 4; j < padded; j += 128) {
    const uint4 k = *reinterpret_cast<const uint4*>(keys + j);
    if (j + 4 <= (int)blockIdx.x * 32) {  // all before in order: equal keys count
      count += (k.x <= key) + (k.y <= key) + (k.z <= key) + (k.w <= key);
    } else if (j >= (int)blockIdx.x * 32 + 32) {
      count += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
    } else {
      count += (k.x < key || (k.x == key && j < me)) + (k.y < key || (k.y == key && j + 1 < me)) +
               (k.z < key || (k.z == key && j + 2 < me)) + (k.w < key || (k.w == key && j + 3 < me));
    }
  }
  before[warp][lane] = count;
  __syncthreads();
  if (warp) return;
  count = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) count += before[w][lane];
  if (me < n) {
    a.key[count] = key;
    a.tok[count] = (uint32_t)me;
  }
}

// Counts of the first pass's digits; those of the passes behind it are set to zero.
__global__ void __launch_bounds__(kBins)
    embed_digit_kernel(const __grid_constant__ EmbedArgs a, const __grid_constant__ SortArgs s) {
  __shared__ uint32_t hist[kBins];
  hist[threadIdx.x] = 0u;
  __syncthreads();
  let_next_begin();
  const int64_t t0 = (int64_t)blockIdx.x * s.tile, t1 = min(t0 + s.tile, a.tokens);
  for (int64_t t = t0 + threadIdx.x; t < t1; t += kBins)
    atomicAdd(&hist[(key_of(a, t) >> s.shift) & ((1u << s.bits) - 1u)], 1u);
  __syncthreads();
  s.count[blockIdx.x * kBins + threadIdx.x] = hist[threadIdx.x];
  for (int p = 1; p <= s.more; ++p) s.count[p * kCounts + blockIdx.x * kBins + threadIdx.x] = 0u;
}

// Sum of v over the threads before this one, and over all (kBins threads).
__device__ __forceinline__ uint32_t scan_bins(uint32_t v, uint32_t* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  uint32_t before = 0;
#pragma unroll
  for (int w = 0; w < kBins / 32; ++w) before += w < warp ? warps[w] : 0u;
  return before + x - v;
}

// A pass: a block finds where its pairs of each digit begin (all blocks'
// smaller digits, earlier blocks' same digits), then moves its pairs in their
// order, kBins at a time; inside a warp equal digits are ranked by lane, warps
// by their order.  The next pass's counts are made on the way (whole numbers:
// their order does not matter).
__global__ void __launch_bounds__(kBins)
    embed_place_kernel(const __grid_constant__ EmbedArgs a, const __grid_constant__ SortArgs s) {
  constexpr int kWarps = kBins / 32;
  __shared__ uint32_t next[kBins], warps[kWarps];
  __shared__ uint16_t wcount[kWarps][kBins];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t mask = (1u << s.bits) - 1u;
  after_previous();
  let_next_begin();
  uint32_t before = 0, total = 0;
#pragma unroll 8
  for (int b = 0; b < s.blocks; ++b) {
    const uint32_t c = __ldcg(s.count + b * kBins + threadIdx.x);
    if (b < (int)blockIdx.x) before += c;
    total += c;
  }
  next[threadIdx.x] = scan_bins(total, warps) + before;
  const int64_t t0 = (int64_t)blockIdx.x * s.tile, t1 = min(t0 + s.tile, a.tokens);
  for (int64_t b = t0; b < t1; b += kBins) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) wcount[w][threadIdx.x] = 0;
    __syncthreads();
    const int64_t t = b + threadIdx.x;
    const bool in = t < t1;
    const uint32_t k = in ? (s.key ? __ldcg(s.key + t) : key_of(a, t)) : 0u;
    const uint32_t d = in ? (k >> s.shift) & mask : kBins;
    const uint32_t same = __match_any_sync(0xffffffffu, d);
    const uint32_t rank = __popc(same & ((1u << lane) - 1u));
    if (in && rank == 0) wcount[warp][d] = (uint16_t)__popc(same);
    __syncthreads();
    uint32_t at = 0;
    if (in) {
      at = next[d] + rank;
      for (int w = 0; w < warp; ++w) at += wcount[w][d];
    }
    __syncthreads();
    uint32_t sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += wcount[w][threadIdx.x];
    next[threadIdx.x] += sum;
    if (in) {
      s.key_out[at] = k;
      s.tok_out[at] = s.tok ? __ldcg(s.tok + t) : (uint32_t)t;
      if (s.more)
        atomicAdd(s.count + kCounts + (at / (uint32_t)s.tile) * kBins +
                      ((k >> (s.shift + s.bits)) & mask),
                  1u);
    }
    __syncthreads();
  }
}

// --- sums ----------------------------------------------------------------------------------------

// A lane's sum of a run to columns c .. of a row (c a multiple of 4).  Added by
// a load and a store: every place is written once in a call.  (Reductions in L2
// would not have to be waited for, but they flush subnormal values to zero.)
template <int V>
__device__ __forceinline__ void put_row(float* row, const float2 (&s)[V / 2], float scale,
                                        int64_t c, int64_t cols, bool add) {
  float v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = __fmul_rn(j & 1 ? s[j / 2].y : s[j / 2].x, scale);
  row += c;
  if ((reinterpret_cast<uintptr_t>(row) & 15u) == 0 && c + V <= cols) {
    if (add) {
      float4 old[V / 4];
#pragma unroll
      for (int j = 0; j < V / 4; ++j) old[j] = __ldcg(reinterpret_cast<const float4*>(row) + j);
#pragma unroll
      for (int j = 0; j < V / 4; ++j) {
        v[4 * j] += old[j].x;
        v[4 * j + 1] += old[j].y;
        v[4 * j + 2] += old[j].z;
        v[4 * j + 3] += old[j].w;
      }
    }
#pragma unroll
    for (int j = 0; j < V; j += 4)
      *reinterpret_cast<float4*>(row + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    return;
  }
  if (add) {
    float old[V];
#pragma unroll
    for (int j = 0; j < V; ++j) old[j] = c + j < cols ? __ldcg(row + j) : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] += old[j];
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (c + j < cols) row[j] = v[j];
}

// Zeros to rows v0 + i of the table, i the bits of `todo`; a warp.
__device__ __forceinline__ void zero_rows(const EmbedArgs& a, int64_t v0, uint32_t todo) {
  const int lane = threadIdx.x & 31;
  while (todo) {
    const int r = __ffs(todo) - 1;
    todo &= todo - 1;
    float* row = a.dtable + (v0 + r) * a.ldd;
    // up to a 16-byte boundary, by 16 bytes, the rest
    const int64_t head =
        min((int64_t)((0u - (uint32_t)(reinterpret_cast<uintptr_t>(row) >> 2)) & 3u), a.cols);
    const int64_t quads = (a.cols - head) >> 2;
    if (lane < head) row[lane] = 0.0f;
    float4* q = reinterpret_cast<float4*>(row + head);
    for (int64_t c = lane; c < quads; c += 32) q[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int64_t c = head + (quads << 2) + lane;
    if (c < a.cols) row[c] = 0.0f;
  }
}

// Few tokens, one launch: every block looks all ids up; a warp has a token and
// 512 bytes of its row, and, where no earlier token has that id, sums the rows
// of all that have it.  The blocks behind them write zeros, 8 rows per warp.
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(256) embed_few_kernel(const __grid_constant__ EmbedArgs a) {
  constexpr int V = Elem<DT>::V, H = V / 2, kDeep = 16;
  __shared__ uint32_t keys[kFew];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = (int)a.tokens;
  const uint32_t none = (uint32_t)a.vocab;
  keys[threadIdx.x] = (int)threadIdx.x < n ? key_of(a, threadIdx.x) : none;
  __syncthreads();
  const int64_t segs = ceil_div(a.row_bytes, (int64_t)512);
  const int64_t sum_blocks = ceil_div(a.tokens * segs, (int64_t)8);
  if (blockIdx.x >= sum_blocks) {
    for (int64_t w = (blockIdx.x - sum_blocks) * 8 + warp; w * 8 < a.vocab;
         w += a.zero_blocks * 8) {
      uint32_t used = 0u;
      for (int j = lane; j < n; j += 32) {
        const uint32_t d = keys[j] - (uint32_t)(w * 8);
        if (d < 8u) used |= 1u << d;
      }
      used = __reduce_or_sync(0xffffffffu, used);
      const int rows = (int)min((int64_t)8, a.vocab - w * 8);
      zero_rows(a, w * 8, ~used & ((1u << rows) - 1u));
    }
    return;
  }
  const int64_t w = (int64_t)blockIdx.x * 8 + warp, t = w / segs;
  if (t >= n) return;
  const uint32_t key = keys[t];
  if (key == none) return;
  for (int j = lane; j < (int)t + lane + 1; j += 32)
    if (__any_sync(0xffffffffu, j < t && keys[j] == key)) return;
  const int64_t off = (w - t * segs) * 512 + lane * 16, c = off / elem_size(DT);
  float2 s[H];
#pragma unroll
  for (int j = 0; j < H; ++j) s[j] = both(0.0f);
  for (int j0 = (int)t & ~31; j0 < n; j0 += 32) {
    uint32_t m = __ballot_sync(0xffffffffu, j0 + lane < n && keys[j0 + lane] == key);
    while (m) {
      uint4 r[kDeep];
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        r[i] = make_uint4(0u, 0u, 0u, 0u);
        if (m)
          r[i] = load_unit<DT, ALIGNED>(a.table + (int64_t)(j0 + __ffs(m) - 1) * a.tpitch, off,
                                        a.row_bytes, a.tend);
        m &= m - 1;
      }
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        float2 v[H];
        unpack2<DT>(r[i], v);
#pragma unroll
        for (int j = 0; j < H; ++j) s[j] = __fadd2_rn(s[j], v[j]);
      }
    }
  }
  put_row<V>(a.dtable + (int64_t)key * a.ldd, s, a.scale, c, a.cols, a.accumulate);
}

// ADD: to what is there, which is brought to L2 while the run is summed (5003
// tokens of 50021 x 1001 fp32, the whole call: 60 -> 56 us).  One kernel for both
// costs 5 us of 166 where nothing is added.
template <int DT, bool ALIGNED, bool ADD>
__global__ void __launch_bounds__(256) embed_sum_kernel(const __grid_constant__ EmbedArgs a) {
  constexpr int V = Elem<DT>::V, H = V / 2, kDeep = 8;
  after_previous();
  let_next_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t chunks = ceil_div(a.tokens, (int64_t)a.chunk);
  const int64_t segs = ceil_div(a.row_bytes, (int64_t)512), seg_blocks = ceil_div(segs, (int64_t)8);
  const int64_t sum_blocks = chunks * seg_blocks;
  if (blockIdx.x >= sum_blocks) {
    // rows without tokens: 8 per warp and round; lanes 0 .. 7 look theirs up
    for (int64_t w = (blockIdx.x - sum_blocks) * 8 + warp; w * 8 < a.vocab;
         w += a.zero_blocks * 8) {
      const int64_t v = w * 8 + (lane & 7);
      int64_t lo = 0, hi = a.tokens;
      while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (__ldg(a.key + mid) < (uint32_t)v) lo = mid + 1;
        else hi = mid;
      }
      const bool empty = lane < 8 && v < a.vocab && (lo == a.tokens || __ldg(a.key + lo) != v);
      zero_rows(a, w * 8, __ballot_sync(0xffffffffu, empty));
    }
    return;
  }
  const int64_t chunk = blockIdx.x / seg_blocks;
  const int64_t seg = (blockIdx.x - chunk * seg_blocks) * 8 + warp;
  if (seg >= segs) return;
  const int64_t p0 = chunk * a.chunk;
  const int n = (int)min((int64_t)a.chunk, a.tokens - p0);
  const int64_t off = seg * 512 + lane * 16, c = off / elem_size(DT);
  // a token's pair per lane, two rounds
  uint32_t key[2], tok[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool in = i * 32 + lane < n;
    key[i] = in ? __ldg(a.key + p0 + i * 32 + lane) : (uint32_t)a.vocab;
    tok[i] = in ? __ldg(a.tok + p0 + i * 32 + lane) : 0u;
  }
  const uint32_t none = (uint32_t)a.vocab;
  const uint32_t before = p0 > 0 ? __ldg(a.key + p0 - 1) : none;
  const uint32_t after = p0 + n < a.tokens ? __ldg(a.key + p0 + n) : none;
  float2 s[H];
#pragma unroll
  for (int j = 0; j < H; ++j) s[j] = both(0.0f);
  uint32_t run = none;  // the id of the run under way
  bool opens = false;   // it began in an earlier chunk
  auto flush = [&](bool goes_on) {
    float* part = a.part + chunk * 2 * a.part_pitch;
    if (opens) put_row<V>(part, s, 1.0f, c, a.cols, false);
    else if (goes_on) put_row<V>(part + a.part_pitch, s, 1.0f, c, a.cols, false);
    else  // (asked again at run time: without that the compiler's code takes 74 us, not 56)
      put_row<V>(a.dtable + (int64_t)run * a.ldd, s, a.scale, c, a.cols, ADD && a.accumulate);
  };
  for (int i0 = 0; i0 < n; i0 += kDeep) {
    uint4 r[kDeep];
    uint32_t k[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      k[i] = __shfl_sync(0xffffffffu, i0 < 32 ? key[0] : key[1], (i0 + i) & 31);
      const uint32_t t = __shfl_sync(0xffffffffu, i0 < 32 ? tok[0] : tok[1], (i0 + i) & 31);
      r[i] = make_uint4(0u, 0u, 0u, 0u);
      if (k[i] != none) {
        r[i] = load_unit<DT, ALIGNED>(a.table + (int64_t)t * a.tpitch, off, a.row_bytes, a.tend);
        // what the run's sum will be added to
        if (ADD && (i == 0 || k[i] != k[i - 1]) && c < a.cols)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(a.dtable + (int64_t)k[i] * a.ldd + c));
      }
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      if (k[i] != run) {
        if (run != none) flush(false);
        run = k[i];
        opens = i0 + i == 0 && run == before;
#pragma unroll
        for (int j = 0; j < H; ++j) s[j] = both(0.0f);
      }
      float2 v[H];
      unpack2<DT>(r[i], v);
#pragma unroll
      for (int j = 0; j < H; ++j) s[j] = __fadd2_rn(s[j], v[j]);
    }
  }
  if (run != none) flush(run == after);
}

// A run that crosses chunks: its first chunk's second partial row, then the
// first ones of the chunks that it goes on in.  A warp per chunk and 128
// columns.
__global__ void __launch_bounds__(256) embed_join_kernel(const __grid_constant__ EmbedArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t chunks = ceil_div(a.tokens, (int64_t)a.chunk);
  const int64_t segs = ceil_div(a.cols, (int64_t)128);
  after_previous();
  const int64_t total = (chunks - 1) * segs, step = (int64_t)gridDim.x * 8;
  const uint32_t none = (uint32_t)a.vocab;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < total; w += step) {
    const int64_t chunk = w / segs;
    const int64_t p0 = chunk * a.chunk, p1 = p0 + a.chunk;
    const uint32_t key = __ldg(a.key + p1 - 1);
    if (key == none || __ldg(a.key + p1) != key) continue;
    if (p0 > 0 && __ldg(a.key + p0 - 1) == key) continue;  // an earlier chunk's run
    const int64_t c = (w - chunk * segs) * 128 + lane * 4;
    // a lane looks at each of the next 32 chunks' first key
    const float* src = a.part + (chunk * 2 + 1) * a.part_pitch + c;
    const bool in = c < a.part_pitch;
    float4 s = in ? *reinterpret_cast<const float4*>(src) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    src += a.part_pitch;
    for (int64_t k = chunk + 1;; k += 32) {
      const int64_t q = (k + lane) * a.chunk;
      const uint32_t on = __ballot_sync(0xffffffffu, q < a.tokens && __ldg(a.key + q) == key);
      const int n = on == 0xffffffffu ? 32 : __ffs(~on) - 1;
      for (int i0 = 0; i0 < n; i0 += 8) {
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = in && i0 + i < n
                     ? *reinterpret_cast<const float4*>(src + (i0 + i) * 2 * a.part_pitch)
                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s.x += v[i].x;
          s.y += v[i].y;
          s.z += v[i].z;
          s.w += v[i].w;
        }
      }
      if (n < 32) break;
      src += 64 * a.part_pitch;
    }
    if (!in) continue;
    const float2 t[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
    put_row<4>(a.dtable + (int64_t)key * a.ldd, t, a.scale, c, a.cols, a.accumulate);
  }
}

// --- host ----------------------------------------------------------------------------------------

int64_t up256(int64_t b) { return round_up(b, 256); }
int64_t part_pitch(int64_t cols) { return round_up(cols, 4); }

// Sorted tokens per unit of work: fewer where there would be fewer warps than
// the GPU takes at once.
int chunk_of(int64_t tokens, int64_t row_bytes) {
  int chunk = kMaxChunk;
  while (chunk > 8 && ceil_div(tokens, (int64_t)chunk) * ceil_div(row_bytes, (int64_t)512) < 2432)
    chunk /= 2;
  return chunk;
}

struct Scratch {
  int64_t key[2], tok[2], count, part, bytes;
};
Scratch lay_out(int64_t tokens, int64_t cols) {
  Scratch s{};
  const bool radix = tokens > kCountMax;
  for (int i = 0; i < (radix ? 2 : 1); ++i) {
    s.key[i] = s.bytes;
    s.bytes += up256(tokens * 4);
    s.tok[i] = s.bytes;
    s.bytes += up256(tokens * 4);
  }
  s.count = s.bytes;
  if (radix) s.bytes += 4 * kCounts * 4;
  s.part = s.bytes;
  // one chunk has no run that crosses
  const int64_t chunks = ceil_div(tokens, (int64_t)chunk_of(tokens, cols * 2));  // 16-bit rows: the most
  if (chunks > 1) s.bytes += chunks * 2 * part_pitch(cols) * 4;
  return s;
}

unsigned warps_grid(const gc_ctx* ctx, int64_t warps, int per_sm) {
  return (unsigned)std::min<int64_t>(ceil_div(warps, (int64_t)8), (int64_t)ctx->num_sms * per_sm);
}

template <int DT, int U>
void lookup_runs(gc_ctx* ctx, const EmbedArgs& a, bool aligned) {
  const unsigned g = warps_grid(ctx, a.tokens * ceil_div(a.row_bytes, (int64_t)(512 * U)), 8);
  if (aligned) embed_forward_kernel<DT, U, true><<<g, 256, 0, ctx->stream>>>(a);
  else embed_forward_kernel<DT, U, false><<<g, 256, 0, ctx->stream>>>(a);
}
// Runs of 2 KB where rows have as many and there is one for every warp that the
// GPU takes (16384 x 4096 bf16: 28 us, by runs of 1 KB 34), of 1 KB elsewhere.
template <int DT>
void lookup(gc_ctx* ctx, const EmbedArgs& a, bool aligned) {
  LaunchScope L(ctx, GC_PHASE_EMBED_FORWARD);
  const bool wide = a.row_bytes >= 2048 && a.tokens * a.row_bytes >= (int64_t)ctx->num_sms * 64 * 2048;
  if (wide) lookup_runs<DT, 4>(ctx, a, aligned);
  else lookup_runs<DT, 2>(ctx, a, aligned);
}
template <int PT, int DT>
void lookup_cast(gc_ctx* ctx, const EmbedArgs& a, bool aligned) {
  using P = typename Elem<PT>::T;
  using T = typename Elem<DT>::T;
  LaunchScope L(ctx, GC_PHASE_EMBED_FORWARD);
  const unsigned g = warps_grid(ctx, a.tokens * ceil_div(a.cols, (int64_t)128), 8);
  if (aligned) embed_cast_kernel<P, T, true><<<g, 256, 0, ctx->stream>>>(a);
  else embed_cast_kernel<P, T, false><<<g, 256, 0, ctx->stream>>>(a);
}

gc_status sort_tokens(gc_ctx* ctx, EmbedArgs& a, char* scratch) {
  const Scratch s = lay_out(a.tokens, a.cols);
  auto at = [&](int64_t o) { return reinterpret_cast<uint32_t*>(scratch + o); };
  if (a.tokens <= kCountMax) {
    a.key = at(s.key[0]);
    a.tok = at(s.tok[0]);
    LaunchScope L(ctx, GC_PHASE_EMBED_SORT);
    embed_count_kernel<<<(unsigned)ceil_div(a.tokens, (int64_t)32), 1024,
                         (size_t)round_up(a.tokens, 128) * 4, ctx->stream>>>(a);
    return GC_OK;
  }
  int bits = 1;
  while (a.vocab >> bits) ++bits;  // keys 0 .. vocab
  const int passes = (bits + 8) / 9;
  SortArgs r{};
  r.bits = (bits + passes - 1) / passes;
  r.tile = (int)round_up(ceil_div(a.tokens, (int64_t)kSortBlocks), kBins);
  r.blocks = (int)ceil_div(a.tokens, (int64_t)r.tile);
  for (int p = 0; p < passes; ++p) {
    const int to = p & 1;
    r.count = at(s.count) + p * kCounts;
    r.shift = p * r.bits;
    r.more = passes - 1 - p;
    if (p == 0) {
      LaunchScope L(ctx, GC_PHASE_EMBED_SORT);
      embed_digit_kernel<<<r.blocks, kBins, 0, ctx->stream>>>(a, r);
    }
    r.key_out = at(s.key[to]);
    r.tok_out = at(s.tok[to]);
    {
      LaunchScope L(ctx, GC_PHASE_EMBED_SORT);
      if (launch_early(embed_place_kernel, dim3(r.blocks), kBins, 0, ctx->stream, a, r) !=
          cudaSuccess)
        return GC_ERR_CUDA;
    }
    r.key = r.key_out;
    r.tok = r.tok_out;
  }
  a.key = r.key_out;
  a.tok = r.tok_out;
  return GC_OK;
}

}  // namespace

int64_t embed_scratch_bytes(int64_t tokens, int64_t vocab, int64_t cols) {
  (void)vocab;
  return tokens == 0 || cols == 0 ? 0 : lay_out(tokens, cols).bytes;
}

gc_status launch_embed_forward(gc_ctx* ctx, const void* ids, int itype, int64_t tokens,
                               int64_t pad, const void* table, int64_t ldtable, int ptype,
                               int64_t vocab, int64_t cols, float scale, void* y, int64_t ldy,
                               int dtype) {
  if (tokens == 0 || cols == 0) return GC_OK;
  EmbedArgs a{};
  a.ids = ids;
  a.wide_ids = itype == GC_I64;
  a.tokens = tokens;
  a.pad = pad;
  a.table = static_cast<const char*>(table);
  a.tpitch = ldtable * elem_size(ptype);
  if (vocab) a.tend = a.table + ((vocab - 1) * ldtable + cols) * elem_size(ptype);
  a.vocab = vocab;
  a.cols = cols;
  a.scale = scale;
  a.y = static_cast<char*>(y);
  a.ypitch = ldy * elem_size(dtype);
  a.row_bytes = cols * elem_size(ptype);
  a.status = ctx->ws.status;
  const bool al = (vocab <= 1 || row_aligned(ldtable, ptype)) && (tokens == 1 || row_aligned(ldy, dtype));
  if (ptype == dtype) {
    if (dtype == GC_F32) lookup<GC_F32>(ctx, a, al);
    else if (dtype == GC_BF16) lookup<GC_BF16>(ctx, a, al);
    else lookup<GC_F16>(ctx, a, al);
  } else {
    if (ptype == GC_F32 && dtype == GC_BF16) lookup_cast<GC_F32, GC_BF16>(ctx, a, al);
    else if (ptype == GC_F32) lookup_cast<GC_F32, GC_F16>(ctx, a, al);
    else if (ptype == GC_BF16 && dtype == GC_F32) lookup_cast<GC_BF16, GC_F32>(ctx, a, al);
    else if (ptype == GC_BF16) lookup_cast<GC_BF16, GC_F16>(ctx, a, al);
    else if (dtype == GC_F32) lookup_cast<GC_F16, GC_F32>(ctx, a, al);
    else lookup_cast<GC_F16, GC_BF16>(ctx, a, al);
  }
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

gc_status launch_embed_wgrad(gc_ctx* ctx, const void* dy, int64_t lddy, int dtype, const void* ids,
                             int itype, int64_t tokens, int64_t pad, int64_t vocab, int64_t cols,
                             float scale, float* dtable, int64_t ldd, int accumulate,
                             void* scratch) {
  if (cols == 0) return GC_OK;
  if (tokens == 0) {
    if (accumulate || vocab == 0) return GC_OK;
    return cudaMemset2DAsync(dtable, ldd * 4, 0, cols * 4, vocab, ctx->stream) == cudaSuccess
               ? GC_OK
               : GC_ERR_CUDA;
  }
  EmbedArgs a{};
  a.ids = ids;
  a.wide_ids = itype == GC_I64;
  a.tokens = tokens;
  a.pad = pad;
  a.table = static_cast<const char*>(dy);
  a.tpitch = lddy * elem_size(dtype);
  a.tend = a.table + ((tokens - 1) * lddy + cols) * elem_size(dtype);
  a.vocab = vocab;
  a.cols = cols;
  a.scale = scale;
  a.dtable = dtable;
  a.ldd = ldd;
  a.accumulate = accumulate;
  a.row_bytes = cols * elem_size(dtype);
  a.status = ctx->ws.status;
  a.part_pitch = part_pitch(cols);
  a.part = reinterpret_cast<float*>(static_cast<char*>(scratch) + lay_out(tokens, cols).part);
  a.chunk = chunk_of(tokens, a.row_bytes);
  const int64_t chunks = ceil_div(tokens, (int64_t)a.chunk);
  const int64_t sum_blocks = chunks * ceil_div(ceil_div(a.row_bytes, (int64_t)512), (int64_t)8);
  a.zero_blocks =
      accumulate ? 0
                 : std::min<int64_t>(ceil_div(vocab, (int64_t)64), (int64_t)ctx->num_sms * 8);
  if (sum_blocks + a.zero_blocks > INT32_MAX) return GC_ERR_UNSUPPORTED;
  const bool al = tokens == 1 || row_aligned(lddy, dtype);
  if (tokens <= kFew) {
    LaunchScope L(ctx, GC_PHASE_EMBED_SUM);
    const auto kernel =
        dtype == GC_F32    ? (al ? embed_few_kernel<GC_F32, true> : embed_few_kernel<GC_F32, false>)
        : dtype == GC_BF16 ? (al ? embed_few_kernel<GC_BF16, true> : embed_few_kernel<GC_BF16, false>)
                           : (al ? embed_few_kernel<GC_F16, true> : embed_few_kernel<GC_F16, false>);
    const int64_t few = ceil_div(tokens * ceil_div(a.row_bytes, (int64_t)512), (int64_t)8);
    if (few + a.zero_blocks > INT32_MAX) return GC_ERR_UNSUPPORTED;
    kernel<<<(unsigned)(few + a.zero_blocks), 256, 0, ctx->stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
  }
  const gc_status st = sort_tokens(ctx, a, static_cast<char*>(scratch));
  if (st != GC_OK) return st;
  {
    LaunchScope L(ctx, GC_PHASE_EMBED_SUM);
    auto pick = [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      return accumulate ? (al ? embed_sum_kernel<DT, true, true> : embed_sum_kernel<DT, false, true>)
                        : (al ? embed_sum_kernel<DT, true, false> : embed_sum_kernel<DT, false, false>);
    };
    const auto kernel = dtype == GC_F32    ? pick(std::integral_constant<int, GC_F32>{})
                        : dtype == GC_BF16 ? pick(std::integral_constant<int, GC_BF16>{})
                                           : pick(std::integral_constant<int, GC_F16>{});
    if (launch_early(kernel, dim3((unsigned)(sum_blocks + a.zero_blocks)), 256, 0, ctx->stream,
                     a) != cudaSuccess)
      return GC_ERR_CUDA;
  }
  if (chunks > 1) {
    LaunchScope L(ctx, GC_PHASE_EMBED_JOIN);
    if (launch_early(embed_join_kernel,
                     dim3(warps_grid(ctx, (chunks - 1) * ceil_div(cols, (int64_t)128), 8)), 256, 0,
                     ctx->stream, a) != cudaSuccess)
      return GC_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

}  // namespace gc
