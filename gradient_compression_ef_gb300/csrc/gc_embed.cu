// gc_embed.cu -- embedding lookup with a scale, and the table's gradient.
//
//   forward   y[t] = scale table[ids[t]]            (pad: zeros)
//   gradient  dtable[v] (+)= scale sum of dy[t] over the tokens t with
//             ids[t] = v, in ascending order of t
//
// The gradient sorts (id, token) pairs, stable, then sums runs of one id:
//   sort      few tokens: each pair's place is the number of pairs before it,
//             counted; more: radix passes of 8 bits (counts, their sums, places)
//   sum       a warp takes 64 sorted tokens and 512 bytes of their rows, and
//             stores each run's sum once: to the table's row where the run lies
//             inside the 64, else to a partial row; warps of their own write
//             zeros to the rows of ids that do not occur
//   join      the partial rows of a run that crosses chunks, in their order
// No atomics on floats: an order of additions that the ids alone decide.
#include <algorithm>
#include <type_traits>

#include "gc_act8.cuh"

namespace gc {
namespace {

constexpr int kChunk = 64;       // sorted tokens of one unit of work
constexpr int kCountMax = 8192;  // tokens that are sorted by counting
constexpr int kTile = 4096;      // tokens of a block of a radix pass

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
  int wide_ids, accumulate;
};

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
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) r[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (row >= 0) {
#pragma unroll
      for (int i = 0; i < U; ++i) r[i] = scale_unit<DT>(r[i], a.scale);
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
  extern __shared__ __align__(16) uint32_t keys[];  // all keys, then the warps' counts
  const int n = (int)a.tokens, padded = (int)round_up(n, 128);
  __shared__ uint32_t before[32][33];
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

// Radix pass, counts: cnt[digit][block] of the blocks' tokens.
__global__ void __launch_bounds__(256)
    embed_digit_kernel(const __grid_constant__ EmbedArgs a, const uint32_t* key, uint32_t* cnt,
                       int64_t blocks, int shift) {
  __shared__ uint32_t hist[256];
  hist[threadIdx.x] = 0u;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  for (int64_t t = t0 + threadIdx.x; t < min(t0 + kTile, a.tokens); t += 256) {
    const uint32_t k = key ? key[t] : key_of(a, t);
    atomicAdd(&hist[(k >> shift) & 255u], 1u);
  }
  __syncthreads();
  cnt[threadIdx.x * blocks + blockIdx.x] = hist[threadIdx.x];
}

// Exclusive sums of cnt: one block per digit sums its row, then places it
// behind the digits before (their totals are counted again: 256 rows).
__global__ void __launch_bounds__(256)
    embed_total_kernel(const uint32_t* cnt, uint32_t* total, int64_t blocks) {
  __shared__ uint32_t s[8];
  uint32_t t = 0;
  for (int64_t b = threadIdx.x; b < blocks; b += 256) t += cnt[blockIdx.x * blocks + b];
#pragma unroll
  for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    t = 0;
    for (int w = 0; w < 8; ++w) t += s[w];
    total[blockIdx.x] = t;
  }
}
__device__ __forceinline__ uint32_t block_scan256(uint32_t v, uint32_t* warps, uint32_t& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  uint32_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    before += w < warp ? warps[w] : 0u;
    all += warps[w];
  }
  return before + x - v;
}
__global__ void __launch_bounds__(256)
    embed_scan_kernel(uint32_t* cnt, const uint32_t* total, int64_t blocks) {
  __shared__ uint32_t warps[8];
  uint32_t all;
  block_scan256(threadIdx.x < blockIdx.x ? total[threadIdx.x] : 0u, warps, all);
  uint32_t base = all;
  for (int64_t b0 = 0; b0 < blocks; b0 += 256) {
    const int64_t b = b0 + threadIdx.x;
    const uint32_t v = b < blocks ? cnt[blockIdx.x * blocks + b] : 0u;
    const uint32_t e = block_scan256(v, warps, all);
    if (b < blocks) cnt[blockIdx.x * blocks + b] = base + e;
    base += all;
  }
}

// Radix pass, places: a block moves its tokens in their order, 256 at a time;
// inside a warp equal digits are ranked by lane, warps by their order.
__global__ void __launch_bounds__(256)
    embed_place_kernel(const __grid_constant__ EmbedArgs a, const uint32_t* key,
                       const uint32_t* tok, const uint32_t* cnt, int64_t blocks, int shift,
                       uint32_t* key_out, uint32_t* tok_out) {
  __shared__ uint32_t next[256], wcount[8][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  next[threadIdx.x] = cnt[threadIdx.x * blocks + blockIdx.x];
  const int64_t t0 = (int64_t)blockIdx.x * kTile, t1 = min(t0 + kTile, a.tokens);
  for (int64_t b = t0; b < t1; b += 256) {
#pragma unroll
    for (int w = 0; w < 8; ++w) wcount[w][threadIdx.x] = 0u;
    __syncthreads();
    const int64_t t = b + threadIdx.x;
    const bool in = t < t1;
    const uint32_t k = in ? (key ? key[t] : key_of(a, t)) : 0u;
    const uint32_t d = in ? (k >> shift) & 255u : 256u;
    const uint32_t same = __match_any_sync(0xffffffffu, d);
    const uint32_t rank = __popc(same & ((1u << lane) - 1u));
    if (in && rank == 0) wcount[warp][d] = __popc(same);
    __syncthreads();
    uint32_t at = 0;
    if (in) {
      at = next[d] + rank;
      for (int w = 0; w < warp; ++w) at += wcount[w][d];
    }
    __syncthreads();
    uint32_t sum = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += wcount[w][threadIdx.x];
    next[threadIdx.x] += sum;
    if (in) {
      key_out[at] = k;
      tok_out[at] = tok ? tok[t] : (uint32_t)t;
    }
    __syncthreads();
  }
}

// --- sums ----------------------------------------------------------------------------------------

// A lane's sum of a run to columns c .. of a row.
template <int V>
__device__ __forceinline__ void put_row(float* row, const float2 (&s)[V / 2], float scale,
                                        int64_t c, int64_t cols, bool add) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float v = __fmul_rn(j & 1 ? s[j / 2].y : s[j / 2].x, scale);
    if (c + j < cols) row[c + j] = add ? row[c + j] + v : v;
  }
}

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(256) embed_sum_kernel(const __grid_constant__ EmbedArgs a) {
  constexpr int V = Elem<DT>::V, H = V / 2, kDeep = 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t chunks = ceil_div(a.tokens, (int64_t)kChunk);
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
      uint32_t todo = __ballot_sync(0xffffffffu, empty);
      while (todo) {
        const int r = __ffs(todo) - 1;
        todo &= todo - 1;
        float* row = a.dtable + (w * 8 + r) * a.ldd;
        // up to a 16-byte boundary, by 16 bytes, the rest
        const int64_t head = min((int64_t)((0u - (uint32_t)(reinterpret_cast<uintptr_t>(row) >> 2)) & 3u), a.cols);
        const int64_t quads = (a.cols - head) >> 2;
        if (lane < head) row[lane] = 0.0f;
        float4* q = reinterpret_cast<float4*>(row + head);
        for (int64_t c = lane; c < quads; c += 32) q[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int64_t c = head + (quads << 2) + lane;
        if (c < a.cols) row[c] = 0.0f;
      }
    }
    return;
  }
  const int64_t chunk = blockIdx.x / seg_blocks;
  const int64_t seg = (blockIdx.x - chunk * seg_blocks) * 8 + warp;
  if (seg >= segs) return;
  const int64_t p0 = chunk * kChunk;
  const int n = (int)min((int64_t)kChunk, a.tokens - p0);
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
    else put_row<V>(a.dtable + (int64_t)run * a.ldd, s, a.scale, c, a.cols, a.accumulate);
  };
  for (int i0 = 0; i0 < n; i0 += kDeep) {
    uint4 r[kDeep];
    uint32_t k[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      k[i] = __shfl_sync(0xffffffffu, i0 < 32 ? key[0] : key[1], (i0 + i) & 31);
      const uint32_t t = __shfl_sync(0xffffffffu, i0 < 32 ? tok[0] : tok[1], (i0 + i) & 31);
      r[i] = make_uint4(0u, 0u, 0u, 0u);
      if (k[i] != none)
        r[i] = load_unit<DT, ALIGNED>(a.table + (int64_t)t * a.tpitch, off, a.row_bytes, a.tend);
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
  const int64_t chunks = ceil_div(a.tokens, (int64_t)kChunk);
  const int64_t segs = ceil_div(a.cols, (int64_t)128);
  after_previous();
  const int64_t total = (chunks - 1) * segs, step = (int64_t)gridDim.x * 8;
  const uint32_t none = (uint32_t)a.vocab;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < total; w += step) {
    const int64_t chunk = w / segs;
    const int64_t p0 = chunk * kChunk, p1 = p0 + kChunk;
    const uint32_t key = __ldg(a.key + p1 - 1);
    if (key == none || __ldg(a.key + p1) != key) continue;
    if (p0 > 0 && __ldg(a.key + p0 - 1) == key) continue;  // an earlier chunk's run
    const int64_t c = (w - chunk * segs) * 128 + lane * 4;
    const float* src = a.part + (chunk * 2 + 1) * a.part_pitch + c;
    if (c >= a.part_pitch) continue;
    float4 s = *reinterpret_cast<const float4*>(src);
    for (int64_t k = chunk + 1; k < chunks; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(a.part + k * 2 * a.part_pitch + c);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
      const int64_t q = (k + 1) * kChunk;
      if (q >= a.tokens || __ldg(a.key + q) != key) break;
    }
    const float2 t[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
    put_row<4>(a.dtable + (int64_t)key * a.ldd, t, a.scale, c, a.cols, a.accumulate);
  }
}

// --- host ----------------------------------------------------------------------------------------

int64_t up256(int64_t b) { return round_up(b, 256); }
int64_t part_pitch(int64_t cols) { return round_up(cols, 4); }

struct Scratch {
  int64_t key[2], tok[2], cnt, total, part, bytes;
};
Scratch lay_out(int64_t tokens, int64_t cols) {
  Scratch s{};
  const int buffers = tokens > kCountMax ? 2 : 1;
  for (int i = 0; i < buffers; ++i) {
    s.key[i] = s.bytes;
    s.bytes += up256(tokens * 4);
    s.tok[i] = s.bytes;
    s.bytes += up256(tokens * 4);
  }
  if (buffers > 1) {
    s.cnt = s.bytes;
    s.bytes += up256(ceil_div(tokens, (int64_t)kTile) * 256 * 4);
    s.total = s.bytes;
    s.bytes += 1024;
  }
  s.part = s.bytes;
  // one chunk has no run that crosses
  if (tokens > kChunk) s.bytes += ceil_div(tokens, (int64_t)kChunk) * 2 * part_pitch(cols) * 4;
  return s;
}

unsigned warps_grid(const gc_ctx* ctx, int64_t warps, int per_sm) {
  return (unsigned)std::min<int64_t>(ceil_div(warps, (int64_t)8), (int64_t)ctx->num_sms * per_sm);
}

template <int DT>
void lookup(gc_ctx* ctx, const EmbedArgs& a, bool aligned) {
  LaunchScope L(ctx, GC_PHASE_EMBED_FORWARD);
  const unsigned g = warps_grid(ctx, a.tokens * ceil_div(a.row_bytes, (int64_t)1024), 8);
  if (aligned) embed_forward_kernel<DT, 2, true><<<g, 256, 0, ctx->stream>>>(a);
  else embed_forward_kernel<DT, 2, false><<<g, 256, 0, ctx->stream>>>(a);
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

void sort_tokens(gc_ctx* ctx, EmbedArgs& a, char* scratch) {
  const Scratch s = lay_out(a.tokens, a.cols);
  auto at = [&](int64_t o) { return reinterpret_cast<uint32_t*>(scratch + o); };
  if (a.tokens <= kCountMax) {
    a.key = at(s.key[0]);
    a.tok = at(s.tok[0]);
    LaunchScope L(ctx, GC_PHASE_EMBED_SORT);
    embed_count_kernel<<<(unsigned)ceil_div(a.tokens, (int64_t)32), 1024,
                         (size_t)round_up(a.tokens, 128) * 4, ctx->stream>>>(a);
    return;
  }
  const int64_t blocks = ceil_div(a.tokens, (int64_t)kTile);
  const uint32_t *key = nullptr, *tok = nullptr;
  int to = 0;
  for (int shift = 0; shift == 0 || (a.vocab >> shift) != 0; shift += 8, to ^= 1) {
    {
      LaunchScope L(ctx, GC_PHASE_EMBED_SORT);
      embed_digit_kernel<<<(unsigned)blocks, 256, 0, ctx->stream>>>(a, key, at(s.cnt), blocks,
                                                                    shift);
    }
    {
      LaunchScope L(ctx, GC_PHASE_EMBED_SORT);
      embed_total_kernel<<<256, 256, 0, ctx->stream>>>(at(s.cnt), at(s.total), blocks);
    }
    {
      LaunchScope L(ctx, GC_PHASE_EMBED_SORT);
      embed_scan_kernel<<<256, 256, 0, ctx->stream>>>(at(s.cnt), at(s.total), blocks);
    }
    {
      LaunchScope L(ctx, GC_PHASE_EMBED_SORT);
      embed_place_kernel<<<(unsigned)blocks, 256, 0, ctx->stream>>>(
          a, key, tok, at(s.cnt), blocks, shift, at(s.key[to]), at(s.tok[to]));
    }
    key = at(s.key[to]);
    tok = at(s.tok[to]);
  }
  a.key = const_cast<uint32_t*>(key);
  a.tok = const_cast<uint32_t*>(tok);
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
  if (vocab == 0 || cols == 0) return GC_OK;
  if (tokens == 0) {
    if (accumulate) return GC_OK;
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
  const int64_t chunks = ceil_div(tokens, (int64_t)kChunk);
  const int64_t sum_blocks = chunks * ceil_div(ceil_div(a.row_bytes, (int64_t)512), (int64_t)8);
  a.zero_blocks =
      accumulate ? 0
                 : std::min<int64_t>(ceil_div(vocab, (int64_t)64), (int64_t)ctx->num_sms * 8);
  if (sum_blocks + a.zero_blocks > INT32_MAX) return GC_ERR_UNSUPPORTED;
  sort_tokens(ctx, a, static_cast<char*>(scratch));
  const bool al = tokens == 1 || row_aligned(lddy, dtype);
  {
    LaunchScope L(ctx, GC_PHASE_EMBED_SUM);
    const auto kernel =
        dtype == GC_F32    ? (al ? embed_sum_kernel<GC_F32, true> : embed_sum_kernel<GC_F32, false>)
        : dtype == GC_BF16 ? (al ? embed_sum_kernel<GC_BF16, true> : embed_sum_kernel<GC_BF16, false>)
                           : (al ? embed_sum_kernel<GC_F16, true> : embed_sum_kernel<GC_F16, false>);
    kernel<<<(unsigned)(sum_blocks + a.zero_blocks), 256, 0, ctx->stream>>>(a);
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
