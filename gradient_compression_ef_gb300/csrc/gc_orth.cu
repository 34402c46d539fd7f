// gc_orth.cu -- an update orthogonalised by Newton-Schulz products.
//
//   X = g / (|g|_F + eps), on its narrow side: [s, l], s = min, l = max of m, n;
//   per step   A = X X^T,  B = a I + b A + c A A,  X <- B X;
//   out = scale X
//
// Every singular value x of X goes to x (a + b x^2 + c x^4) in each step and
// the singular vectors stay.  Directions far below the largest one grow by a
// factor of a each step, and so do errors in them, so that the iterates carry
// 22 bits: each is held as two fp16 planes, v 2^12 = hi + lo 2^-11, and a product
// is hi hi + 2^-11 (hi lo + lo hi) on the tensor cores (tcgen05, exact products,
// fp32 accumulation; lo lo is below 2^-22 and left out).  The products with lo
// come first, and the first hi hi multiplies the sum so far by 2^-11.  Magnitudes:
// X, A and B of a converging polynomial stay below 16; small entries keep their
// digits down to 2^-48 absolute, half of fp16's smallest step in lo.  (With v 2^12
// = hi + lo that was 2^-37: a row of an update 10^8 times below another one came
// out to 5e-3 of its size.)
//
// An update far below eps makes X far below 1: X is 2^e times its planes, one e <=
// 0 for the whole matrix and step, from a bound r on its largest singular value,
// r_0 = |g| / (|g| + eps), r <- r (|a| + |b| r^2 + |c| r^4).  From a bound of 1/2 on
// e is 0.  The powers of two are put in when sums are stored.
//
// An input in 16 bits is held in one plane, times the power of two that brings
// its largest element to 2^14 .. 2^15 (what X_0 is beyond that is one more factor,
// f, put in likewise): the first step's A takes one product, its B X two.  That is
// exact for elements down to 2^-31 (bf16) or 2^-28 (fp16) of the largest; those
// below are held to 2^-39 of it.
//
// The result's type decides the last rounding alone: a bf16 result is the fp32
// one, rounded.  (X and B of the last step with 11 bits took 13 % off 11008 x
// 4096 bf16, but where few singular directions carry the update their roundings
// are coherent, and add as much as the rounding to bf16.)
//
// A and B are symmetric: tiles below the diagonal are not computed, what lies
// above it is stored twice, mirrored.  a is put on B's diagonal, so that
// a step's last product needs no epilogue.
//
// A product: one persistent CTA pair per two SMs (cta_group::2) owns tiles of
// 256 x TN.  Blocks of 64 of the sum's axis come by TMA (128-byte swizzle),
// both planes of both operands; each block is 12 MMAs.
//   producer   one warp: TMA
//   issuer     one warp of the leader CTA: the MMAs of the pair
//   read-out   8 warps: tensor memory -> running sums in registers -> planes
// The tensor cores round their running sums towards zero; read-out takes them
// over block by block and adds in registers, rounded to nearest.  (By two or four
// blocks: 2 and 4 % faster, with two and five times the error.)
//
// Measured: 4096 x 4096 fp32, five steps 2830 to 2920 us from card to card (4.12
// Tflop in fp16 products: 1410 to 1460 Tflop/s; cuBLAS bf16 1912 for a burst,
// 1698 sustained): the board's power limit lowers the clock to 1.75 GHz within a
// product, where a block of 256 x 256 x 64 x 3 takes 0.897 us, 98 % of what that
// clock gives; the rest is the last round's idle pairs and a tile's epilogue, 3
// to 5 us.  11008 x 4096 bf16 5730 to 5900 us (8.60 Tflop).  1001 x 2051: 233 to
// 238 us, 15 dependent launches of 13 us, a third of it on the tensor cores.  128
// x 64: 29 us in one kernel.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "gc_act8.cuh"
#include "gc_sm100.cuh"

namespace gc {
namespace {

constexpr int kTM = 256;             // rows of a pair's tile
constexpr int kBK = 64;              // of the sum's axis, per block
constexpr uint32_t kABytes = 128 * kBK * 2;  // one plane, one CTA
constexpr int kReadWarps = 8, kProducerWarp = 8, kIssuerWarp = 9;
constexpr int kThreads = 384;
// Registers a thread: as launched, and (tiles of 256 columns) of the read-out
// warps and of the other four; 8 * 232 + 4 * 40 = 12 * 168.
constexpr int kLaunchRegs = 168, kReadRegs = 232, kOtherRegs = 40;
static_assert(8 * kReadRegs + 4 * kOtherRegs <= 12 * kLaunchRegs);
constexpr long long kWaitCycles = 4000000000ll;  // bound on each wait: ~2 s
constexpr uint32_t kWarpStage = 4096;  // of a read-out warp, for its stores
constexpr int kMaxPartsOfTile = 4, kMaxPairs = 80;
constexpr int kMaxParts = 608;       // blocks of the norm's kernel
constexpr float kUnit = 4096.0f;     // planes hold v * kUnit
constexpr int kLoBits = 11;          // the second plane's units are so many bits smaller
constexpr float kLo = 1 << kLoBits;

enum { kGram = 0, kPoly = 1, kApply = 2, kLast = 3 };

// What a step's planes stand for: X = f 2^e times them (over kUnit).
struct Range {
  float gram;   // f^2 4^e: of A's sums
  float apply;  // f 2^(e - the next step's e): of B X's, written by A's kernel
  float f;
  float unit;   // 2^e
  float r;      // bound on X's largest singular value
  int e;
};
// The power of two that holds values up to r, from -126 to 0; a NaN's is 0.
__device__ __forceinline__ int exponent_of(float r) {
  return r < 0.5f ? (int)(__float_as_uint(r) >> 23) - 126 : 0;
}
__device__ __forceinline__ float power2(int e) {  // of -126 .. 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
__device__ __forceinline__ Range make_range(float f, float r, int e) {
  const float unit = power2(e);
  return {f * f * unit * unit, 0.0f, f, unit, r, e};
}
// The bound after a step; what A's kernel writes: the next step's range and the
// factor of B X.
__device__ __forceinline__ float grown(float r, float a, float b, float c) {
  const float q = r * r;
  return r * fmaf(q, fmaf(q, fabsf(c), fabsf(b)), fabsf(a));
}
__device__ __forceinline__ void next_range(Range* now, Range* next, float a, float b, float c) {
  const float r = grown(__ldcg(&now->r), a, b, c);
  const int e = exponent_of(r);
  now->apply = __ldcg(&now->f) * power2(__ldcg(&now->e) - e);
  *next = make_range(1.0f, r, e);
}

// What a sum over a block of 16 k elements loses on average to the tensor
// cores' roundings towards zero, as a share of its value: put back when it is
// read.  Measured as the mean of sum(x^2) - 1 over unit vectors x; in B X,
// whose sums have one large term (B is near a multiple of the identity), as
// the shrinking of a step's result, about half of it in whole blocks.
__host__ __device__ constexpr float lost(int k, int mode) {
  return (k >= 4 ? 3.0f : k == 3 ? 2.2f : k == 2 ? 1.5f : 0.9f) *
         (k >= 4 && (mode == kApply || mode == kLast) ? 0x1p-25f : 0x1p-24f);
}

template <int TN>
struct Shape {
  static constexpr int kBN = TN / 2;                       // second operand, one CTA
  static constexpr uint32_t kBBytes = kBN * kBK * 2;       // one plane
  static constexpr uint32_t kStage = 2 * (kABytes + kBBytes);
  static constexpr int kStages = TN == 256 ? 3 : 4;
  static constexpr uint32_t kCols = 2 * TN;                // tensor memory: two accumulators
  static constexpr size_t kSmem =
      1024 + (size_t)kStages * kStage + kReadWarps * kWarpStage + 8 * (2 * kStages + 5) + 16;
};

struct ProductArgs {
  int64_t rows, cols;      // of the result
  int64_t sum;             // length of the sum
  int64_t row_tiles, col_tiles;
  int64_t whole, items;    // tiles computed whole; all items of work
  int parts;               // the tiles behind them are computed in so many parts
  float* part;             // sums of the parts, [split tile][part][CTA of the pair][..]
  uint32_t* arrived;       // [split tile][CTA of the pair][warp], zero before and after
  uint16_t* dst;           // planes of the result, plane_size apart
  const uint16_t* prev;    // kPoly: A's planes
  int64_t pitch, plane_size;  // elements
  int a_planes, b_planes;  // of the operands: 2, or their first alone
  Range *range, *next_range;  // of this step and of the next
  float a, b, c;
  void* out;               // kLast
  int64_t ldo;
  float scale;
  int odtype, transposed, out_vec;
  uint32_t* status;
};

struct Smem {
  uint32_t stage0, out0;
  uint64_t *full, *empty, *acc_full, *acc_empty, *drain;
  uint32_t* tmem_slot;
  float* factors;  // of the sums, of the result
};
template <int TN>
__device__ __forceinline__ Smem carve(unsigned char* base) {
  using S = Shape<TN>;
  Smem s;
  const uint32_t at = (sm100::smem_u32(base) + 1023u) & ~1023u;
  unsigned char* p = base + (at - sm100::smem_u32(base));
  s.stage0 = at;
  s.out0 = at + S::kStages * S::kStage;
  s.full = reinterpret_cast<uint64_t*>(p + S::kStages * S::kStage + kReadWarps * kWarpStage);
  s.empty = s.full + S::kStages;
  s.acc_full = s.empty + S::kStages;
  s.acc_empty = s.acc_full + 2;
  s.drain = s.acc_empty + 2;
  s.tmem_slot = reinterpret_cast<uint32_t*>(s.drain + 1);
  s.factors = reinterpret_cast<float*>(s.tmem_slot + 1);
  return s;
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int32_t x,
                                                 int32_t y, int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// v = hi + lo / kLo as two fp16 values each, of a pair: hi the nearest, lo the
// nearest to the rest.
__device__ __forceinline__ void split2(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(v0, v1);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(__fsub_rn(v0, f.x) * kLo, __fsub_rn(v1, f.y) * kLo);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ float2 join2(uint32_t hi, uint32_t lo) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  const float2 l = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  return make_float2(fmaf(l.x, 1.0f / kLo, h.x), fmaf(l.y, 1.0f / kLo, h.y));
}

// Tiles by rows of tiles, outputs of neighbouring columns next to one another;
// of a symmetric result those on and above the diagonal.
template <int TN, bool SYM>
__device__ __forceinline__ void tile_place(const ProductArgs& a, int64_t t, int64_t& i, int64_t& j) {
  if (!SYM) {
    // bands of 8 row tiles, rows fastest: the tiles that pairs work on at the
    // same time share their operands in L2
    const int64_t per = 8 * a.col_tiles, band = t / per, r = t - band * per;
    const int64_t w = min((int64_t)8, a.row_tiles - band * 8);
    j = r / w;
    i = band * 8 + r - j * w;
    return;
  }
  for (i = 0;; ++i) {
    const int64_t first = i * kTM / TN, n = a.col_tiles - first;
    if (t < n) {
      j = first + t;
      return;
    }
    t -= n;
  }
}

template <int DT>
__device__ __forceinline__ void put(void* out, int64_t at, float v) {
  if (DT == GC_F32) static_cast<float*>(out)[at] = v;
  else if (DT == GC_BF16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[at] = __float2half_rn(v);
}

// Item t of the work: a tile and the blocks [k0, k1) of its sum.  Tiles go
// round by round; those that would leave most pairs idle in a last round are
// computed in parts of the sum.
template <int TN, bool SYM>
struct Item {
  int64_t i, j, split;  // split: which of the tiles in parts, or -1
  int32_t k0, k1;
  int part;
  __device__ __forceinline__ Item(const ProductArgs& a, int64_t t, int32_t blocks) {
    split = -1;
    part = 0;
    k0 = 0;
    k1 = blocks;
    if (t >= a.whole) {
      if (a.parts > 1) {
        split = (t - a.whole) / a.parts;
        part = (int)(t - a.whole - split * a.parts);
        k0 = blocks * part / a.parts;
        k1 = blocks * (part + 1) / a.parts;
        t = a.whole + split;
      }
    }
    tile_place<TN, SYM>(a, t, i, j);
  }
};

// Where 16 bytes c of row r lie in a warp's stage of 32 rows of 128 bytes: no
// bank is hit twice when lanes write a row each, when 8 lanes read a row, and
// when rows 8 q + 2 m, 8 q + 2 m + 1 (q = 0 .. 3) are read as a matrix.
__device__ __forceinline__ uint32_t staged(uint32_t stage, int r, int c) {
  return stage + (uint32_t)r * 128u + (uint32_t)((c ^ (r & 7) ^ ((r >> 3) << 1)) << 4);
}
__device__ __forceinline__ void sts_u128(uint32_t at, uint32_t x, uint32_t y, uint32_t z,
                                         uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z),
               "r"(w)
               : "memory");
}
// Column lane / 4 of 8, rows 8 (lane % 4) .. + 7 of the stage's 32, of the
// fp16 elements of 16 bytes c.
__device__ __forceinline__ uint4 staged_column(uint32_t stage, int c) {
  const int lane = threadIdx.x & 31;
  // lane 8 m + k names row k of matrix m
  const int m = lane >> 3, k = lane & 7;
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(staged(stage, (k >> 1) * 8 + 2 * m + (k & 1), c))
               : "memory");
  return v;
}

// One plane of 64 columns from j on of the warp's 32 rows from i on, staged,
// and of a symmetric result their mirror image: a group of 8 columns of a row
// that lies below the diagonal to its last element is the mirror's, every other
// one the row's own, so that each element is written once.  (Short code: a
// tile's epilogue runs once or a few times in a kernel, and fetching its
// instructions was half of its time.)
template <bool SYM>
__device__ __forceinline__ void store_plane(const ProductArgs& a, uint16_t* dst, uint32_t stage,
                                            int64_t i, int64_t j) {
  const int lane = threadIdx.x & 31;
  const int rows = (int)min((int64_t)32, a.rows - i), cols = (int)min((int64_t)64, a.cols - j);
  const int d = (int)min((int64_t)64, j - i);  // >= -63
  uint16_t* p = dst + (i + (lane >> 3)) * a.pitch + j + (lane & 7) * 8;
#pragma unroll
  for (int k = 0; k < 8; ++k, p += 4 * a.pitch) {
    const int r = k * 4 + (lane >> 3), c = (lane & 7) * 8;
    const uint4 v = sm100::lds_u128(staged(stage, r, lane & 7));
    // rows of planes are padded to whole groups of 8
    if (r < rows && c < cols && (!SYM || c + 7 + d >= r)) *reinterpret_cast<uint4*>(p) = v;
  }
  if (!SYM) return;
  p = dst + (j + (lane >> 2)) * a.pitch + i + (lane & 3) * 8;
#pragma unroll
  for (int k = 0; k < 8; ++k, p += 8 * a.pitch) {
    const int r = (lane & 3) * 8, c = k * 8 + (lane >> 2);
    const uint4 v = staged_column(stage, k);
    if (c < cols && r + 7 < c + d) *reinterpret_cast<uint4*>(p) = v;
  }
}

// A warp's part of an output of type DT, rows from i, columns from j on, by
// rows: through the stage, 128 bytes of each row at a time.
template <int DT, int N>
__device__ __forceinline__ void store_rows(const ProductArgs& a, const float (&v)[N], float scale,
                                           uint32_t stage, int64_t i, int64_t j) {
  constexpr int E = elem_size(DT), C = 128 / E, V = Elem<DT>::V;
  using T = typename Elem<DT>::T;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c0 = 0; c0 < N; c0 += C) {
    if (j + c0 >= a.cols) break;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float u[V];
#pragma unroll
      for (int e = 0; e < V; ++e) u[e] = __fmul_rn(v[c0 + k * V + e], scale);
      const uint4 r = Elem<DT>::pack(u);
      sts_u128(staged(stage, lane, k), r.x, r.y, r.z, r.w);
    }
    __syncwarp();
    if (a.out_vec) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t r = i + k * 4 + (lane >> 3), c = j + c0 + (lane & 7) * V;
        if (r >= a.rows || c >= a.cols) continue;
        const uint4 q = sm100::lds_u128(staged(stage, k * 4 + (lane >> 3), lane & 7));
        char* p = reinterpret_cast<char*>(static_cast<T*>(a.out) + r * a.ldo + c);
        if (c + V <= a.cols) *reinterpret_cast<uint4*>(p) = q;
        else store_some<DT>(p, q, 0, (int)(a.cols - c));
      }
    } else {
#pragma unroll 4
      for (int r = 0; r < 32; ++r) {
        if (i + r >= a.rows) break;
        T* p = static_cast<T*>(a.out) + (i + r) * a.ldo + j + c0;
#pragma unroll
        for (int h = 0; h < C / 32; ++h) {
          const int c = h * 32 + lane;
          if (j + c0 + c >= a.cols) continue;
          const uint32_t at = staged(stage, r, c / V) + (uint32_t)(c % V) * E;
          if constexpr (E == 4) {
            reinterpret_cast<uint32_t*>(p)[c] = sm100::lds_u32(at);
          } else {
            uint16_t q;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(q) : "r"(at) : "memory");
            reinterpret_cast<uint16_t*>(p)[c] = q;
          }
        }
      }
    }
  }
}
template <int DT, int N>
__device__ __forceinline__ void store_result(const ProductArgs& a, const float (&v)[N],
                                             float scale, uint32_t stage, int64_t i, int64_t j) {
  if (!a.transposed) {
    store_rows<DT, N>(a, v, scale, stage, i, j);
    return;
  }
  const int64_t r = i + (threadIdx.x & 31);
  if (r >= a.rows) return;
#pragma unroll
  for (int c = 0; c < N; ++c)
    if (j + c < a.cols) put<DT>(a.out, (j + c) * a.ldo + r, __fmul_rn(v[c], scale));
}

// A warp's part of a tile, 32 rows from i, N columns from j on, from the sums.
template <int MODE, int N>
__device__ __forceinline__ void store_tile(const ProductArgs& a, float (&sum)[N],
                                           const float* factors, uint32_t stage, int64_t i,
                                           int64_t j) {
  constexpr bool kSym = MODE == kGram || MODE == kPoly;
  const int lane = threadIdx.x & 31;
  if (i >= a.rows) return;
  const float unit = MODE == kPoly ? 1.0f / kUnit : factors[0];
#pragma unroll
  for (int c = 0; c < N; ++c) sum[c] = fmaf(sum[c], lost(kBK / 16, MODE), sum[c]) * unit;
  if (MODE == kLast) {
    const float scale = factors[1];
    if (a.odtype == GC_F32) store_result<GC_F32, N>(a, sum, scale, stage, i, j);
    else if (a.odtype == GC_BF16) store_result<GC_BF16, N>(a, sum, scale, stage, i, j);
    else store_result<GC_F16, N>(a, sum, scale, stage, i, j);
    return;
  }
#pragma unroll
  for (int c0 = 0; c0 < N; c0 += 64) {
    const int64_t jc = j + c0;
    if (jc >= a.cols || (kSym && jc + 63 < i)) continue;  // outside, or the mirror's
    if (MODE == kPoly) {
#pragma unroll
      for (int e = 0; e < 64; ++e) sum[c0 + e] *= a.c;
      // plus b A, read by rows, both planes at once
      const uint16_t* src = a.prev + (i + (lane >> 3)) * a.pitch + jc + (lane & 7) * 8;
      const bool in = jc + (lane & 7) * 8 < a.cols;
      uint4 q[2][8];
#pragma unroll
      for (int k = 0; k < 8; ++k, src += 4 * a.pitch) {
        q[0][k] = q[1][k] = make_uint4(0u, 0u, 0u, 0u);
        if (in && i + k * 4 + (lane >> 3) < a.rows) {
          q[0][k] = __ldcg(reinterpret_cast<const uint4*>(src));
          q[1][k] = __ldcg(reinterpret_cast<const uint4*>(src + a.plane_size));
        }
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          sts_u128(staged(stage, k * 4 + (lane >> 3), lane & 7), q[p][k].x, q[p][k].y, q[p][k].z,
                   q[p][k].w);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float2 f[4];
          unpack2<GC_F16>(sm100::lds_u128(staged(stage, lane, k)), f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float b = p ? a.b * (1.0f / kLo) : a.b;
            float* t = sum + c0 + k * 8 + 2 * e;
            t[0] = fmaf(b, f[e].x, t[0]);
            t[1] = fmaf(b, f[e].y, t[1]);
          }
        }
      }
      if (jc < i + 32) {  // the diagonal comes through
        const int64_t d = i + lane - jc;
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (e == d) sum[c0 + e] += a.a * kUnit;
      }
    }
    // the first planes; what is left of the values are the second ones
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float* t = sum + c0 + k * 8 + 2 * e;
        const __half2 w = __floats2half2_rn(t[0], t[1]);
        const float2 f = __half22float2(w);
        t[0] = __fsub_rn(t[0], f.x);
        t[1] = __fsub_rn(t[1], f.y);
        h[e] = *reinterpret_cast<const uint32_t*>(&w);
      }
      sts_u128(staged(stage, lane, k), h[0], h[1], h[2], h[3]);
    }
    __syncwarp();
    store_plane<kSym>(a, a.dst, stage, i, jc);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t l[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* t = sum + c0 + k * 8 + 2 * e;
        const __half2 w = __floats2half2_rn(t[0] * kLo, t[1] * kLo);
        l[e] = *reinterpret_cast<const uint32_t*>(&w);
      }
      sts_u128(staged(stage, lane, k), l[0], l[1], l[2], l[3]);
    }
    __syncwarp();
    store_plane<kSym>(a, a.dst + a.plane_size, stage, i, jc);
  }
}

// A part's sums go to the scratch; the warp that comes last adds all parts, in
// their order, and has the tile.
template <int N>
__device__ __forceinline__ bool join_parts(const ProductArgs& a, float (&sum)[N], int64_t split,
                                           int part, uint32_t rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto at = [&](int p) {
    return reinterpret_cast<float4*>(a.part) +
           (((split * a.parts + p) * 2 + rank) * kReadWarps + warp) * (N / 4 * 32) + lane;
  };
  float4* mine = at(part);
#pragma unroll
  for (int c = 0; c < N; c += 4)
    __stcg(mine + c * 8, make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]));
  __threadfence();
  __syncwarp();
  uint32_t* count = a.arrived + (split * 2 + rank) * kReadWarps + warp;
  uint32_t before = 0;
  if (lane == 0) before = atomicAdd(count, 1u);
  before = __shfl_sync(0xffffffffu, before, 0);
  if (before != (uint32_t)a.parts - 1u) return false;
  __threadfence();
  if (lane == 0) *count = 0u;  // as it was, for the next product
#pragma unroll
  for (int c = 0; c < N; ++c) sum[c] = 0.0f;
  for (int p = 0; p < a.parts; ++p) {
    const float4* src = at(p);
    constexpr int kBatch = 16;  // loads in flight
#pragma unroll
    for (int c0 = 0; c0 < N; c0 += 4 * kBatch) {
      float4 f[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) f[k] = __ldcg(src + (c0 + 4 * k) * 8);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        float* t = sum + c0 + 4 * k;
        t[0] += f[k].x;
        t[1] += f[k].y;
        t[2] += f[k].z;
        t[3] += f[k].w;
      }
    }
  }
  return true;
}

template <int MODE, int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    orth_product_kernel(const __grid_constant__ CUtensorMap map_a,
                        const __grid_constant__ CUtensorMap map_b,
                        const __grid_constant__ ProductArgs a) {
  using namespace sm100;
  using S = Shape<TN>;
  constexpr bool kSym = MODE == kGram || MODE == kPoly;
  constexpr bool kBMN = !kSym;  // the second operand's columns lie contiguous
  extern __shared__ unsigned char orth_smem[];
  const Smem s = carve<TN>(orth_smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int32_t blocks = (int32_t)((a.sum + kBK - 1) / kBK);
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], 2 * kReadWarps);
    }
    mbar_init(s.drain, 1);
    mbar_fence_init();
  }
  if (warp == kIssuerWarp) {
    tmem_alloc_pair(s.tmem_slot, S::kCols);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // the pair's barriers exist before either CTA arrives on one
  tc_fence_after_sync();
  const uint32_t tmem = *s.tmem_slot;
  bool ok = true;
  let_next_begin();
  if (warp < kReadWarps) {
    if constexpr (TN == 256) reg_inc<kReadRegs>();
    // warp w reads lanes 32 (w % 4) .. + 31 (rows) of columns N (w / 4) .. of
    // every accumulator
    constexpr int N = TN / 2;
    const uint32_t q = (uint32_t)warp & 3u, ch = (uint32_t)warp >> 2;
    const uint32_t acc_empty0 = map_to_rank(smem_u32(s.acc_empty), 0);
    after_previous();
    // fetched while the first blocks come, kept in shared memory (every warp
    // writes the same for itself)
    if (MODE != kPoly && lane == 0) {
      if (MODE == kGram) s.factors[0] = __ldcg(&a.range->gram) * (1.0f / kUnit);
      if (MODE == kApply) s.factors[0] = __ldcg(&a.range->apply) * (1.0f / kUnit);
      if (MODE == kLast) {
        s.factors[0] = __ldcg(&a.range->f) * (1.0f / (kUnit * kUnit));
        s.factors[1] = a.scale * __ldcg(&a.range->unit);
      }
    }
    __syncwarp();
    uint32_t seg = 0;
    for (int64_t t = pair; ok && t < a.items; t += pairs) {
      const Item<TN, kSym> item(a, t, blocks);
      float sum[N];
#pragma unroll
      for (int c = 0; c < N; ++c) sum[c] = 0.0f;
      for (int32_t k = item.k0; k < item.k1; ++k, ++seg) {
        const uint32_t buf = seg & 1u;
        const bool got = mbar_wait_cluster(&s.acc_full[buf], (seg >> 1) & 1u, kWaitCycles);
        if (__any_sync(0xffffffffu, !got)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t at = tmem + ((q * 32) << 16) + buf * TN + ch * N;
#pragma unroll
        for (int j = 0; j < N / 16; ++j) {
          float v[16];
          tmem_ld16(at + j * 16, v);
#pragma unroll
          for (int c = 0; c < 16; ++c) sum[j * 16 + c] += v[c];
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty0 + buf * 8);
      }
      if (!ok) break;
      if (item.split < 0 || join_parts<N>(a, sum, item.split, item.part, rank))
        store_tile<MODE, N>(a, sum, s.factors, s.out0 + warp * kWarpStage,
                            item.i * kTM + rank * 128 + q * 32, item.j * TN + ch * N);
      __syncwarp();
    }
  } else {
    if constexpr (TN == 256) reg_dec<kOtherRegs>();
    if (warp == kProducerWarp) {
      const uint32_t bar0 = map_to_rank(smem_u32(s.full), 0);  // the leader counts the bytes
      const uint32_t stage_bytes = 2 * (a.a_planes * kABytes + a.b_planes * S::kBBytes);
      after_previous();
      int st = 0;
      uint32_t ph = 0, loads = 0;
      for (int64_t t = pair; ok && t < a.items; t += pairs) {
        const Item<TN, kSym> item(a, t, blocks);
        const int32_t r0 = (int32_t)(item.i * kTM) + (int32_t)rank * 128;
        const int32_t c0 = (int32_t)(item.j * TN) + (int32_t)rank * S::kBN;
        for (int32_t k = item.k0; k < item.k1; ++k) {
          if (loads >= S::kStages) {
            // free once the pair's MMAs read it
            if (!mbar_wait_cluster(&s.empty[st], ph ^ 1u, kWaitCycles)) ok = false;
            if (__any_sync(0xffffffffu, !ok)) {
              ok = false;
              break;
            }
          } else {
            ++loads;
          }
          if (elect_one()) {
            const uint32_t bar = bar0 + st * 8, at = s.stage0 + st * S::kStage;
            if (rank == 0) mbar_arrive_expect_tx(&s.full[st], stage_bytes);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              if (p < a.a_planes)
                tma_load_3d_pair(at + p * kABytes, &map_a, k * kBK, r0, p, bar);
              if (p >= a.b_planes) continue;
              const uint32_t b = at + 2 * kABytes + p * S::kBBytes;
              if (!kBMN) {
                tma_load_3d_pair(b, &map_b, k * kBK, c0, p, bar);
              } else {
#pragma unroll
                for (int h = 0; h < S::kBN / 64; ++h)
                  tma_load_3d_pair(b + h * 8192, &map_b, c0 + h * 64, k * kBK, p, bar);
              }
            }
          }
          if (++st == S::kStages) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
      // the arrivals of the last MMAs on this CTA's barriers: none may be under
      // way when the CTA ends
      for (int i = 0; ok && i < S::kStages; ++i) {
        if (loads >= S::kStages || (uint32_t)st < loads)
          if (!mbar_wait_cluster(&s.empty[st], ph ^ 1u, kWaitCycles)) ok = false;
        if (++st == S::kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
    } else if (warp == kIssuerWarp) {
      if (rank == 0) {
        constexpr uint32_t idesc = (1u << 4) | ((kBMN ? 1u : 0u) << 16) |
                                   ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(kTM >> 4) << 24);
        // K-major: 128-byte rows of 64, 8 rows per 1024-byte group; 16 of the sum
        // are 32 bytes.  MN-major: 128-byte rows of 64 columns, 8 of the sum per
        // group, blocks of 64 columns 8 KB apart; 16 of the sum are 2048 bytes.
        const uint64_t da = smem_desc_sw128(s.stage0, 16, 1024);
        const uint64_t db = smem_desc_sw128(s.stage0 + 2 * kABytes, kBMN ? 8192 : 16, 1024);
        const uint32_t hi = (uint32_t)(da >> 32), a0 = (uint32_t)da, b0 = (uint32_t)db;
        constexpr uint32_t kAStep = 32 >> 4, kBStep = (kBMN ? 2048 : 32) >> 4;
        constexpr uint32_t kALo = kABytes >> 4, kBLo = S::kBBytes >> 4;
        int st = 0;
        uint32_t ph = 0, seg = 0;
        for (int64_t t = pair; ok && t < a.items; t += pairs) {
          const Item<TN, kSym> item(a, t, blocks);
          for (int32_t k = item.k0; k < item.k1; ++k, ++seg) {
            const uint32_t buf = seg & 1u;
            if (seg >= 2 &&
                !mbar_wait_cluster(&s.acc_empty[buf], ((seg >> 1) - 1u) & 1u, kWaitCycles))
              ok = false;
            if (ok && !mbar_wait_cluster(&s.full[st], ph, kWaitCycles)) ok = false;
            if (__any_sync(0xffffffffu, !ok)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            if (elect_one()) {
              const uint32_t off = (uint32_t)st * (S::kStage >> 4), d = tmem + buf * TN;
              // the products with lo first, kLoBits ahead of the others (a block
              // has the accumulator to itself)
              uint32_t more = 0u;
              auto multiply = [&](uint32_t a_at, uint32_t b_at) {
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk) {
                  mma_f16_pair(d, a0 + off + a_at + kk * kAStep, b0 + off + b_at + kk * kBStep, hi,
                               idesc, more);
                  more = 1u;
                }
              };
              if (a.a_planes == 2) multiply(kALo, 0u);
              if (a.b_planes == 2) multiply(0u, kBLo);
              if (more) mma_f16_pair_behind<kLoBits>(d, a0 + off, b0 + off, hi, idesc);
              else mma_f16_pair(d, a0 + off, b0 + off, hi, idesc, 0u);
#pragma unroll
              for (int kk = 1; kk < kBK / 16; ++kk)
                mma_f16_pair(d, a0 + off + kk * kAStep, b0 + off + kk * kBStep, hi, idesc, 1u);
              mma_commit_pair(&s.empty[st]);
              mma_commit_pair(&s.acc_full[buf]);
            }
            if (++st == S::kStages) {
              st = 0;
              ph ^= 1u;
            }
          }
        }
        if (elect_one()) mma_commit_pair(s.drain);
      }
    } else if (MODE == kGram && blockIdx.x == 0 && warp == kIssuerWarp + 1 && lane == 0) {
      after_previous();
      next_range(a.range, a.next_range, a.a, a.b, a.c);
    }
  }
  // MMAs still in flight read both CTAs' shared memory: the producers, which
  // have kept step with them as far as here, wait for the issuer's last commit
  if (warp == kProducerWarp && ok && !mbar_wait_cluster(s.drain, 0, kWaitCycles)) ok = false;
  if (!ok) {
    atomicOr(a.status, kStatusWaitTimeout);
    // a wait ran out: let copies in flight land before the CTA's memory goes
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000ll) {
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == kIssuerWarp) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, S::kCols);
  }
}

// --- norm and planes of g ------------------------------------------------------------------------

struct InputArgs {
  const void* g;
  int64_t m, n, ld;      // as given
  int64_t pitch, plane_size;
  double* part;          // sums of squares, one per block
  int parts;
  float eps;
  uint16_t* dst;
  uint32_t* top;         // the blocks' largest magnitudes, as bits (16-bit types)
  Range* range;          // of X_0
  uint32_t* arrived;     // the products' counters, set to zero
};

template <int DT>
__device__ __forceinline__ float get(const void* g, int64_t at) {
  if (DT == GC_F32) return __ldg(static_cast<const float*>(g) + at);
  if (DT == GC_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(g)[at]);
  return __half2float(static_cast<const __half*>(g)[at]);
}

// Eight consecutive elements of a row, zero from column n on.  VEC: rows start
// on 16-byte boundaries.
template <int DT, bool VEC>
__device__ __forceinline__ void get8(float (&v)[8], const InputArgs& a, int64_t r, int64_t c) {
  if (VEC && c + 8 <= a.n) {
    const char* p = static_cast<const char*>(a.g) + (r * a.ld + c) * elem_size(DT);
    if constexpr (DT == GC_F32) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p));
      const float4 y = __ldg(reinterpret_cast<const float4*>(p) + 1);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
      v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    } else {
      Elem<DT>::unpack(__ldg(reinterpret_cast<const uint4*>(p)), v);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = c + e < a.n ? get<DT>(a.g, r * a.ld + c + e) : 0.0f;
}

// Sum of N times eight squares: in fp32 where they keep clear of its range's
// ends, in binary64 (a small fraction of fp32's rate) where not.
template <int N>
__device__ __forceinline__ double sum_squares(const float (&v)[N][8]) {
  float top = 0.0f, q[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    q[k] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      top = fmaxf(top, fabsf(v[k][e]));
      q[k] = fmaf(v[k][e], v[k][e], q[k]);
    }
  }
#pragma unroll
  for (int h = 1; h < N; h *= 2)
#pragma unroll
    for (int k = 0; k + h < N; k += 2 * h) q[k] += q[k + h];
  if (top == 0.0f || (top > 0x1p-50f && top < 0x1p58f)) return (double)q[0];
  double t = 0.0;
  for (int k = 0; k < N; ++k)
    for (int e = 0; e < 8; ++e) t += (double)v[k][e] * (double)v[k][e];
  return t;
}

// X_0's factor: kUnit / (|g| + eps) = n 2^(e - k), where 2^e holds r = |g| / (|g| +
// eps).  The sum of squares is m 4^k with 1 <= m < 4, so that root and quotient
// are fp32 ones (binary64's take thousands of cycles).  n = 0 where g is zero (or
// eps beyond binary32's range times it), NaN where g is not finite.
struct Unit {
  float n, r;
  int k, e;
  __device__ __forceinline__ Unit(double squares, float eps) : n(0.0f), r(0.0f), k(0), e(0) {
    if (squares == 0.0) return;
    if (!(squares <= 1.0e300)) {
      n = NAN;
      return;
    }
    const long long bits = __double_as_longlong(squares);
    const int x = (int)(bits >> 52) - 1023;
    k = x >> 1;
    const float m = (float)__longlong_as_double((bits & 0xFFFFFFFFFFFFFll) |
                                                ((long long)(1023 + x - 2 * k) << 52));
    const float root = sqrtf(m), t = root + ldexpf(eps, -k);
    r = root / t;
    e = exponent_of(r);
    n = kUnit / t * power2(-e);
  }
  // of g's elements, for planes that stand for 2^e times them: as two factors,
  // each inside binary32's range whatever the norm
  __device__ __forceinline__ float2 factors() const {
    return make_float2(ldexpf(1.0f, -(k / 2)), ldexpf(n, -(k - k / 2)));
  }
};

// Segment `seg` of 256 columns of row r, every `step`-th of all: without a
// division for each.
struct Walk {
  int64_t r, seg, segs, step_r, step_seg;
  __device__ __forceinline__ Walk(int64_t first, int64_t step, int64_t segs_)
      : r(first / segs_), seg(first - r * segs_), segs(segs_), step_r(step / segs_),
        step_seg(step - step_r * segs_) {}
  __device__ __forceinline__ void next() {
    r += step_r;
    seg += step_seg;
    if (seg >= segs) {
      seg -= segs;
      ++r;
    }
  }
};

// Sums of squares, a double per block.
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) orth_norm_kernel(const __grid_constant__ InputArgs a) {
  __shared__ double s[8];
  __shared__ uint32_t tops[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t segs = ceil_div(a.n, (int64_t)256);
  double sum = 0.0;
  uint32_t top = 0u;
  let_next_begin();
  if (blockIdx.x == 0)
    for (int k = threadIdx.x; k < kMaxPairs * 2 * kReadWarps; k += 256) a.arrived[k] = 0u;
  Walk at((int64_t)blockIdx.x * 8 + warp, (int64_t)gridDim.x * 8, segs);
  while (at.r < a.m) {
    float v[4][8];  // four loads on their way
#pragma unroll
    for (int k = 0; k < 4; ++k, at.next())
      get8<DT, VEC>(v[k], a, at.r, at.r < a.m ? at.seg * 256 + lane * 8 : a.n);
    sum += sum_squares<4>(v);
    if (DT != GC_F32) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[k][e]) & 0x7FFFFFFFu);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (DT != GC_F32) top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) {
    s[warp] = sum;
    tops[warp] = top;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int w = 0; w < 8; ++w) {
      t += s[w];
      top = max(top, tops[w]);
    }
    a.part[blockIdx.x] = t;
    if (DT != GC_F32) a.top[blockIdx.x] = top;
  }
}

// What g's elements are multiplied by, from the blocks' sums; the whole block
// calls it, and the first one writes X_0's range.  fp32: Unit's factors.  16-bit
// types: the power of two that brings the largest magnitude to 2^14 .. 2^15, the
// rest being the range's f.
template <int DT>
__device__ __forceinline__ float2 plane_factors(const InputArgs& a) {
  __shared__ float2 f;
  if (threadIdx.x < 32) {
    double t = 0.0;
    uint32_t top = 0u;
    double d[kMaxParts / 32];
#pragma unroll
    for (int k = 0; k < kMaxParts / 32; ++k) {
      const int p = k * 32 + threadIdx.x;
      d[k] = p < a.parts ? a.part[p] : 0.0;
      if (DT != GC_F32 && p < a.parts) top = max(top, a.top[p]);
    }
#pragma unroll
    for (int k = 0; k < kMaxParts / 32; ++k) t += d[k];
#pragma unroll
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (DT != GC_F32) top = __reduce_max_sync(0xffffffffu, top);
    if (threadIdx.x == 0) {
      const Unit u(t, a.eps);
      float rest = 1.0f;
      if (DT == GC_F32) {
        f = u.factors();
      } else {
        const bool some = u.n > 0.0f;  // neither zero nor NaN
        const int p = some ? 14 - ilogbf(__uint_as_float(top)) : 0;
        f = make_float2(ldexpf(1.0f, p / 2), ldexpf(1.0f, p - p / 2));
        rest = some ? ldexpf(u.n, -u.k - p) : u.n;
      }
      if (blockIdx.x == 0) *a.range = make_range(rest, u.r, u.e);
    }
  }
  __syncthreads();
  return f;
}

// A zero times NaN is NaN: not finite anywhere makes NaN everywhere.
__device__ __forceinline__ float in_units(float v, float2 f) {
  return __fmul_rn(__fmul_rn(v, f.x), f.y);
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(256) orth_split_kernel(const __grid_constant__ InputArgs a) {
  after_previous();
  let_next_begin();
  const float2 f = plane_factors<DT>(a);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (Walk at((int64_t)blockIdx.x * 8 + warp, (int64_t)gridDim.x * 8, ceil_div(a.n, (int64_t)256));
       at.r < a.m; at.next()) {
    const int64_t r = at.r, c = at.seg * 256 + lane * 8;
    if (c >= a.n) continue;
    float v[8];
    get8<DT, VEC>(v, a, r, c);
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      split2(in_units(v[2 * e], f), in_units(v[2 * e + 1], f), h[e], l[e]);
    uint16_t* dst = a.dst + r * a.pitch + c;
    *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
    if (DT == GC_F32)
      *reinterpret_cast<uint4*>(dst + a.plane_size) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

// The same for m > n, transposed: tiles of 64 x 64 through shared memory.
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) orth_turn_kernel(const __grid_constant__ InputArgs a) {
  __shared__ float t[64][65];
  after_previous();
  let_next_begin();
  const float2 f = plane_factors<DT>(a);
  const int64_t ct = ceil_div(a.n, (int64_t)64), total = ceil_div(a.m, (int64_t)64) * ct;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int64_t r0 = w / ct * 64, c0 = (w % ct) * 64;
    __syncthreads();
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = h * 256 + threadIdx.x;
      const int64_t r = r0 + (k >> 3);
      if (r < a.m) get8<DT, VEC>(v[h], a, r, c0 + (k & 7) * 8);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = h * 256 + threadIdx.x;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        t[k >> 3][(k & 7) * 8 + e] = r0 + (k >> 3) < a.m ? in_units(v[h][e], f) : 0.0f;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < 64 * 8; k += 256) {
      const int c = k >> 3, r = (k & 7) * 8;
      if (c0 + c >= a.n || r0 + r >= a.m) continue;
      uint32_t h[4], l[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(t[r + 2 * e][c], t[r + 2 * e + 1][c], h[e], l[e]);
      uint16_t* dst = a.dst + (c0 + c) * a.pitch + r0 + r;
      *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
      if (DT == GC_F32)
        *reinterpret_cast<uint4*>(dst + a.plane_size) = make_uint4(l[0], l[1], l[2], l[3]);
    }
  }
}

// --- narrow matrices: every step in one kernel --------------------------------------------------
//
// s <= 128: a CTA keeps 256 columns of X in shared memory for the whole call
// (both planes; the layout is the same whether the sum runs along a row, in X
// X^T, or along a column, in B X), and A, then B, in one buffer.  Several CTAs
// (a cooperative launch) add their parts of A through L2: each adds up its
// share of the elements, then all read A.  A barrier takes about 1.5 us.

constexpr int kSmallS = 128, kSmallCols = 256, kSmallSteps = 32;
constexpr uint32_t kBlock = 128 * 128;  // 128 rows of 64 columns, one plane
constexpr uint32_t kXPlane = (kSmallCols / 64) * kBlock, kAPlane = 2 * kBlock;
constexpr size_t kSmallSmem = 1024 + 2 * kXPlane + 2 * kAPlane;

struct SmallArgs {
  const void* g;
  void* out;
  int64_t l, ldg, ldo;
  int s, s16, tall, dtype, odtype, steps;
  float eps, scale;
  double* norms;     // [CTAs]
  float* part;       // [CTAs][s16][s16]
  uint32_t* gram;    // [s16][s16], hi | lo << 16
  uint32_t* arrived;
  uint32_t* status;
  float coefs[kSmallSteps][3];
};

// Elements (i, j .. j + 7) of X's slice, j a multiple of 8; zero outside.
template <int DT>
__device__ __forceinline__ void get_slice(float (&v)[8], const SmallArgs& a, int i, int64_t j) {
  const int64_t at = a.tall ? j * a.ldg + i : i * a.ldg + j, step = a.tall ? a.ldg : 1;
  if (i < a.s && j + 8 <= a.l) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = get<DT>(a.g, at + e * step);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = i < a.s && j + e < a.l ? get<DT>(a.g, at + e * step) : 0.0f;
  }
}

// Place of 16 bytes (row i, columns 8 c ..) in a plane of blocks of 64 columns.
__device__ __forceinline__ uint32_t chunk_at(int i, int c) {
  return (uint32_t)(c >> 3) * kBlock + (uint32_t)i * 128u + (uint32_t)(((c ^ i) & 7) << 4);
}
__device__ __forceinline__ void put_planes(uint32_t at, uint32_t plane, const float (&v)[8]) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) split2(v[2 * e], v[2 * e + 1], h[e], l[e]);
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(h[0]), "r"(h[1]),
               "r"(h[2]), "r"(h[3])
               : "memory");
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + plane), "r"(l[0]), "r"(l[1]),
               "r"(l[2]), "r"(l[3])
               : "memory");
}

// Row r and columns 8 c .. of the slice that a thread takes in its w-th turn:
// neighbouring lanes along the axis that is contiguous in memory.
__device__ __forceinline__ void slice_place(const SmallArgs& a, int chunks, int w, int& r, int& c) {
  r = a.tall ? w % a.s16 : w / chunks;
  c = a.tall ? w / a.s16 : w % chunks;
}

// The slice's sum of squares (a thread's part); the elements are kept at `hold`
// (shared memory), if that is not 0, in fp32.  (Loops that are not unrolled: in
// a kernel that runs once through its code, fetching the code counts.)
template <int DT>
__device__ __forceinline__ double slice_squares(const SmallArgs& a, int64_t c0, int chunks,
                                                uint32_t hold) {
  const int total = a.s16 * chunks;
  double sum = 0.0;
#pragma unroll 1
  for (int w0 = threadIdx.x; w0 < total; w0 += 4 * 256) {
    float v[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      int r, c;
      slice_place(a, chunks, w0 + k * 256, r, c);
      get_slice<DT>(v[k], a, r, c0 + c * 8);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int w = w0 + k * 256;
      if (w >= total) {  // another slice's, or nothing
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] = 0.0f;
      } else if (hold) {
        sm100::sts128(hold + w * 32, make_float4(v[k][0], v[k][1], v[k][2], v[k][3]));
        sm100::sts128(hold + w * 32 + 16, make_float4(v[k][4], v[k][5], v[k][6], v[k][7]));
      }
    }
    sum += sum_squares<4>(v);
  }
  return sum;
}

// The slice, in units, to its planes.
template <int DT>
__device__ __forceinline__ void slice_planes(const SmallArgs& a, int64_t c0, int chunks, float2 f,
                                             uint32_t xs, uint32_t hold) {
#pragma unroll 1
  for (int w = threadIdx.x; w < a.s16 * chunks; w += 256) {
    int r, c;
    slice_place(a, chunks, w, r, c);
    float v[8];
    if (hold) {
      const float4 p = sm100::lds128(hold + w * 32), q = sm100::lds128(hold + w * 32 + 16);
      v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w;
      v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
    } else {
      get_slice<DT>(v, a, r, c0 + c * 8);
    }
    const int64_t left = r < a.s ? a.l - c0 - c * 8 : 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? in_units(v[e], f) : 0.0f;
    put_planes(xs + chunk_at(r, c), kXPlane, v);
  }
}

// 16 columns of a row of the result.
template <int DT>
__device__ __forceinline__ void put_slice(const SmallArgs& a, int i, int64_t j,
                                          const float (&v)[16], float scale) {
  const int64_t at = a.tall ? j * a.ldo + i : i * a.ldo + j, step = a.tall ? a.ldo : 1;
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (j + e < a.l)
      put<DT>(a.out, at + e * step, __fmul_rn(v[e] * (1.0f / kUnit), scale));
}

// Every CTA of the grid is here, and what it wrote is visible; false when the
// wait ran out.
__device__ __forceinline__ bool grid_barrier(const SmallArgs& a, uint32_t& target) {
  __shared__ uint32_t ok;
  __syncthreads();
  target += gridDim.x;
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(a.arrived, 1u);
    const long long t0 = clock64();
    uint32_t n;
    do {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(a.arrived) : "memory");
    } while (n < target && clock64() - t0 < kWaitCycles);
    ok = n >= target;
  }
  __syncthreads();
  return ok != 0u;
}

// The MMAs of a product: `blocks` blocks of 64 of the sum (the last of `tail`
// 16s), each into an accumulator of its own, 512 / accumulators columns apart.
template <bool MN>
__device__ __forceinline__ void small_product(uint32_t tmem, uint32_t cols, uint32_t a_at,
                                              uint32_t a_plane, uint32_t b_at, uint32_t b_plane,
                                              int sixteens, uint32_t idesc) {
  using namespace sm100;
  const uint64_t da = smem_desc_sw128(a_at, 16, 1024);
  const uint64_t db = smem_desc_sw128(b_at, MN ? kBlock : 16, 1024);
  const uint32_t hi = (uint32_t)(da >> 32), a0 = (uint32_t)da, b0 = (uint32_t)db;
  // 16 of the sum: 32 bytes of a row, every 64 the next block; or 16 rows
  auto a_step = [](int k) { return ((uint32_t)(k >> 2) * kBlock + (uint32_t)(k & 3) * 32u) >> 4; };
  auto b_step = [&](int k) { return MN ? ((uint32_t)k * 2048u) >> 4 : a_step(k); };
  for (int k0 = 0; k0 < sixteens; k0 += 4) {
    const uint32_t d = tmem + (uint32_t)(k0 >> 2) * cols;
    const int k1 = min(k0 + 4, sixteens);
    for (int k = k0; k < k1; ++k)
      mma_f16_one(d, a0 + (a_plane >> 4) + a_step(k), b0 + b_step(k), hi, idesc, k > k0);
    for (int k = k0; k < k1; ++k)
      mma_f16_one(d, a0 + a_step(k), b0 + (b_plane >> 4) + b_step(k), hi, idesc, 1u);
    mma_f16_one_behind<kLoBits>(d, a0 + a_step(k0), b0 + b_step(k0), hi, idesc);
    for (int k = k0 + 1; k < k1; ++k)
      mma_f16_one(d, a0 + a_step(k), b0 + b_step(k), hi, idesc, 1u);
  }
}

__global__ void __launch_bounds__(256, 1) orth_small_kernel(const __grid_constant__ SmallArgs a) {
  using namespace sm100;
  extern __shared__ unsigned char small_smem[];
  __shared__ uint64_t done;
  __shared__ uint32_t tmem_slot;
  __shared__ double norm_part[8];
  __shared__ float2 factors;
  __shared__ float bound;  // on X_0's largest singular value
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t xs = (smem_u32(small_smem) + 1023u) & ~1023u, as = xs + 2 * kXPlane;
  const int64_t c0 = (int64_t)blockIdx.x * kSmallCols;
  const int cols = (int)min((int64_t)kSmallCols, a.l - c0);
  const int x16 = (cols + 15) / 16, xpad = x16 * 16;
  const uint32_t row0 = (uint32_t)(warp & 3) * 32u;
  const int i = (int)row0 + lane, half = warp >> 2;
  const bool mine = i < a.s16;
  uint32_t target = 0, phase = 0;
  bool ok = true;
  if (threadIdx.x == 0) {
    mbar_init(&done, 1);
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }

  // the slice's sum of squares
  const int chunks = xpad / 8;
  // A's place holds g's slice until the planes are made, where it fits
  const uint32_t hold = a.s16 * xpad * 4 <= (int)(2 * kAPlane) ? as : 0u;
  double sum = a.dtype == GC_F32    ? slice_squares<GC_F32>(a, c0, chunks, hold)
               : a.dtype == GC_BF16 ? slice_squares<GC_BF16>(a, c0, chunks, hold)
                                    : slice_squares<GC_F16>(a, c0, chunks, hold);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) norm_part[warp] = sum;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) {
      sum = 0.0;
      for (int w = 0; w < 8; ++w) sum += norm_part[w];
      a.norms[blockIdx.x] = sum;
    }
    ok = grid_barrier(a, target);
  }
  if (warp == 0) {
    sum = 0.0;
    if (gridDim.x > 1)
      for (int p = lane; p < (int)gridDim.x; p += 32) sum += __ldcg(a.norms + p);
    else if (lane < 8)
      sum = norm_part[lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      const Unit u(sum, a.eps);
      factors = u.factors();
      bound = u.r;
    }
  }
  __syncthreads();
  const float2 f = factors;
  float r = bound;
  if (a.dtype == GC_F32) slice_planes<GC_F32>(a, c0, chunks, f, xs, hold);
  else if (a.dtype == GC_BF16) slice_planes<GC_BF16>(a, c0, chunks, f, xs, hold);
  else slice_planes<GC_F16>(a, c0, chunks, f, xs, hold);

  auto idesc = [](int n, bool mn) {
    return (1u << 4) | ((mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
  };
  // Operands are in place; issues a product and waits for it.
  auto multiply = [&](int what) {
    fence_proxy_async_smem();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0 && elect_one()) {
      const int s = a.s16 / 16;
      if (what == kGram)
        small_product<false>(tmem, 128, xs, kXPlane, xs, kXPlane, x16, idesc(a.s16, false));
      else if (what == kPoly)
        small_product<false>(tmem, 128, as, kAPlane, as, kAPlane, s, idesc(a.s16, false));
      else
        small_product<true>(tmem, 256, as, kAPlane, xs, kXPlane, s, idesc(xpad, true));
      mma_commit(&done);
    }
    __syncwarp();
    if (!mbar_wait(&done, phase, kWaitCycles)) ok = false;
    phase ^= 1u;
    tc_fence_after_sync();
  };
  // 16 columns from c on of this thread's row, from `parts` accumulators, in units.
  auto take = [&](float (&v)[16], int c, int mode, int sixteens, uint32_t apart, float unit) {
    const int parts = (sixteens + 3) / 4;
    const float back = lost(sixteens, mode);
    tmem_ld16(tmem + (row0 << 16) + c, v);
    for (int p = 1; p < parts; ++p) {
      float w[16];
      tmem_ld16(tmem + (row0 << 16) + p * apart + c, w);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] += w[e];
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = fmaf(v[e], back, v[e]) * unit;
  };
  auto store16 = [&](uint32_t at, uint32_t plane, int c, const float (&v)[16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = v[h * 8 + e];
      put_planes(at + chunk_at(i, (c >> 3) + h), plane, u);
    }
  };

  for (int step = 0; step < a.steps && ok; ++step) {
    multiply(kGram);
    // X is 2^e times its planes, and 2^next the next one
    const int e = exponent_of(r);
    r = grown(r, a.coefs[step][0], a.coefs[step][1], a.coefs[step][2]);
    const int next = exponent_of(r);
    const float unit = power2(e);
    for (int c = half * 16; c < a.s16; c += 32) {
      float v[16];
      take(v, c, kGram, x16, 128, unit * unit * (1.0f / kUnit));
      if (!mine) continue;
      if (gridDim.x == 1) {
        store16(as, kAPlane, c, v);
      } else {
        float* p = a.part + ((int64_t)blockIdx.x * a.s16 + c) * a.s16 + i;
#pragma unroll
        for (int e = 0; e < 16; ++e) __stcg(p + e * a.s16, v[e]);
      }
    }
    if (gridDim.x > 1) {
      const int all = a.s16 * a.s16;
      if (!grid_barrier(a, target)) ok = false;
      for (int e = blockIdx.x * 256 + threadIdx.x; e < all; e += gridDim.x * 256) {
        float v = 0.0f;
#pragma unroll 8
        for (int p = 0; p < (int)gridDim.x; ++p) v += __ldcg(a.part + (int64_t)p * all + e);
        uint32_t h, l;
        split2(v, 0.0f, h, l);
        __stcg(a.gram + e, (h & 0xFFFFu) | (l << 16));
      }
      if (!grid_barrier(a, target)) ok = false;
      for (int q = threadIdx.x; q < all / 8; q += 256) {
        const uint4 u = __ldcg(reinterpret_cast<const uint4*>(a.gram) + 2 * q);
        const uint4 w = __ldcg(reinterpret_cast<const uint4*>(a.gram) + 2 * q + 1);
        const int r = q * 8 / a.s16, c = q * 8 - r * a.s16;
        const uint32_t at = as + chunk_at(r, c >> 3);
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                     "r"(__byte_perm(u.x, u.y, 0x5410)), "r"(__byte_perm(u.z, u.w, 0x5410)),
                     "r"(__byte_perm(w.x, w.y, 0x5410)), "r"(__byte_perm(w.z, w.w, 0x5410))
                     : "memory");
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + kAPlane),
                     "r"(__byte_perm(u.x, u.y, 0x7632)), "r"(__byte_perm(u.z, u.w, 0x7632)),
                     "r"(__byte_perm(w.x, w.y, 0x7632)), "r"(__byte_perm(w.z, w.w, 0x7632))
                     : "memory");
      }
    }
    multiply(kPoly);
    const float ca = a.coefs[step][0] * kUnit, cb = a.coefs[step][1], cc = a.coefs[step][2];
    for (int c = half * 16; c < a.s16; c += 32) {
      float v[16];
      take(v, c, kPoly, a.s16 / 16, 128, 1.0f / kUnit);
      if (!mine) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = as + chunk_at(i, (c >> 3) + h);
        const uint4 hi = lds_u128(at), lo = lds_u128(at + kAPlane);
        const uint32_t hw[4] = {hi.x, hi.y, hi.z, hi.w}, lw[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 p = join2(hw[e], lw[e]);
          const int k = h * 8 + 2 * e;
          v[k] = fmaf(cc, v[k], cb * p.x);
          v[k + 1] = fmaf(cc, v[k + 1], cb * p.y);
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (c + e == i) v[e] += ca;
      store16(as, kAPlane, c, v);
    }
    multiply(kApply);
    const bool last = step + 1 == a.steps;
    const float to_next = (last ? 1.0f : power2(e - next)) * (1.0f / kUnit);
    ok = !__syncthreads_or(!ok);  // a wait that ran out ends the call for every thread
    for (int c = half * 16; c < xpad; c += 32) {
      float v[16];
      take(v, c, kApply, a.s16 / 16, 256, to_next);
      if (!mine) continue;
      if (!last) {
        store16(xs, kXPlane, c, v);
      } else if (i < a.s) {
        if (a.odtype == GC_F32) put_slice<GC_F32>(a, i, c0 + c, v, a.scale * unit);
        else if (a.odtype == GC_BF16) put_slice<GC_BF16>(a, i, c0 + c, v, a.scale * unit);
        else put_slice<GC_F16>(a, i, c0 + c, v, a.scale * unit);
      }
    }
  }
  if (!ok) atomicOr(a.status, kStatusWaitTimeout);
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// --- host ----------------------------------------------------------------------------------------



PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

// A matrix as two fp16 planes in the scratch.
struct Planes {
  uint16_t* at;
  int64_t rows, cols, pitch, size;  // size: elements of a plane
};
int64_t plane_pitch(int64_t cols) { return round_up(cols, 64); }
int64_t planes_bytes(int64_t rows, int64_t cols) { return 2 * rows * plane_pitch(cols) * 2; }

bool make_map(CUtensorMap* map, const Planes& p, uint32_t box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)p.cols, (cuuint64_t)p.rows, 2};
  const cuuint64_t strides[2] = {(cuuint64_t)(p.pitch * 2), (cuuint64_t)(p.size * 2)};
  const cuuint32_t boxes[3] = {kBK, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, p.at, dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How T tiles are dealt to the pairs, and what that costs in cycles, as measured:
// a block of 64 of the sum, a tile's epilogue, a part's way through memory and
// its share of the joining, for tiles of 256 and of 128 columns.
struct Deal {
  int64_t whole, items;
  int parts;
  double cost;
};
Deal deal(int64_t tiles, int64_t pairs, int64_t blocks, int tn, int products) {
  const double block = (tn == 256 ? 1540 : 820) * products / 3.0, store = tn == 256 ? 7000 : 4500;
  const double leave = tn == 256 ? 5000 : 4000, join = tn == 256 ? 2200 : 1300;
  const int64_t full = tiles / pairs * pairs, rem = tiles - full;
  Deal d{tiles, tiles, 1, (double)ceil_div(tiles, pairs) * ((double)blocks * block + store)};
  if (!rem) return d;
  for (int p = 2; p <= std::min<int64_t>({pairs / rem, kMaxPartsOfTile, blocks}); ++p) {
    const double cost = (double)(full / pairs) * ((double)blocks * block + store) +
                        (double)ceil_div(blocks, (int64_t)p) * block + leave + p * join + store;
    if (cost < d.cost) d = {full, full + rem * p, p, cost};
  }
  return d;
}

// Tiles of a [rows, cols] result; of a symmetric one those on and above the
// diagonal.
int64_t count_tiles(int64_t rows, int64_t cols, int tn, bool sym) {
  const int64_t r = ceil_div(rows, (int64_t)kTM), c = ceil_div(cols, (int64_t)tn);
  if (!sym) return r * c;
  int64_t n = 0;
  for (int64_t i = 0; i < r; ++i) n += c - i * kTM / tn;
  return n;
}

template <int MODE, int TN>
gc_status product(gc_ctx* ctx, const Planes& x, const Planes& y, const Planes& d, ProductArgs a,
                  const Deal& deal) {
  static uint64_t devices = 0;
  constexpr bool kSym = MODE == kGram || MODE == kPoly;
  if (!allow_smem(ctx, orth_product_kernel<MODE, TN>, (int)Shape<TN>::kSmem, devices))
    return GC_ERR_CUDA;
  // the registers that warps take over have to be there
  static const bool regs = [] {
    cudaFuncAttributes f{};
    return TN != 256 || (cudaFuncGetAttributes(&f, orth_product_kernel<MODE, TN>) == cudaSuccess &&
                         f.numRegs >= kLaunchRegs);
  }();
  if (!regs) return GC_ERR_CUDA;
  CUtensorMap ma, mb;
  if (!make_map(&ma, x, 128) || !make_map(&mb, y, kSym ? TN / 2 : kBK)) return GC_ERR_CUDA;
  a.rows = d.rows;
  a.cols = d.cols;
  a.sum = x.cols;
  a.row_tiles = ceil_div(d.rows, (int64_t)kTM);
  a.col_tiles = ceil_div(d.cols, (int64_t)TN);
  a.whole = deal.whole;
  a.items = deal.items;
  a.parts = deal.parts;
  a.dst = d.at;
  a.pitch = d.pitch;
  a.plane_size = d.size;
  a.status = ctx->ws.status;
  const int64_t pairs = std::min<int64_t>(a.items, ctx->num_sms / 2);
  LaunchScope L(ctx, GC_PHASE_ORTH_PRODUCT);
  return launch_early(orth_product_kernel<MODE, TN>, dim3((unsigned)(2 * pairs)), kThreads,
                      Shape<TN>::kSmem, ctx->stream, ma, mb, a) == cudaSuccess
             ? GC_OK
             : GC_ERR_CUDA;
}

template <int MODE>
gc_status product(gc_ctx* ctx, const Planes& x, const Planes& y, const Planes& d,
                  const ProductArgs& a) {
  constexpr bool kSym = MODE == kGram || MODE == kPoly;
  const int64_t pairs = std::min(ctx->num_sms / 2, kMaxPairs), blocks = ceil_div(x.cols, (int64_t)kBK);
  const int products = a.a_planes + a.b_planes - 1;
  const Deal wide = deal(count_tiles(d.rows, d.cols, 256, kSym), pairs, blocks, 256, products);
  const Deal slim = deal(count_tiles(d.rows, d.cols, 128, kSym), pairs, blocks, 128, products);
  return slim.cost < wide.cost ? product<MODE, 128>(ctx, x, y, d, a, slim)
                               : product<MODE, 256>(ctx, x, y, d, a, wide);
}

// Scratch of the tiles in parts: at most kMaxPairs items of work, and no more
// than kMaxPartsOfTile for each tile, of 256 columns or of twice as many of 128.
int64_t parts_bytes(int64_t s, int64_t l) {
  const int64_t tiles = count_tiles(s, l, 256, false);
  return std::min<int64_t>(kMaxPairs, kMaxPartsOfTile * tiles) * kTM * 256 * 4;
}
constexpr int64_t kTopBytes = kMaxParts * 4 + 256;  // and two ranges
static_assert(2 * sizeof(Range) <= 256);
constexpr int64_t kArrivedBytes = kMaxPairs * 2 * kReadWarps * 4;

template <int DT>
gc_status input(gc_ctx* ctx, const InputArgs& a) {
  const bool vec = (reinterpret_cast<uintptr_t>(a.g) & 15u) == 0 && (a.m == 1 || row_aligned(a.ld, DT));
  {
    LaunchScope L(ctx, GC_PHASE_ORTH_INPUT);
    const auto k = vec ? orth_norm_kernel<DT, true> : orth_norm_kernel<DT, false>;
    k<<<a.parts, 256, 0, ctx->stream>>>(a);
  }
  LaunchScope L(ctx, GC_PHASE_ORTH_INPUT);
  cudaError_t e;
  if (a.m > a.n) {
    const int64_t tiles = ceil_div(a.m, (int64_t)64) * ceil_div(a.n, (int64_t)64);
    const dim3 g((unsigned)std::min<int64_t>(tiles, (int64_t)ctx->num_sms * 8));
    e = vec ? launch_early(orth_turn_kernel<DT, true>, g, 256, 0, ctx->stream, a)
            : launch_early(orth_turn_kernel<DT, false>, g, 256, 0, ctx->stream, a);
  } else {
    const int64_t warps = a.m * ceil_div(a.n, (int64_t)256);
    const dim3 g((unsigned)std::min<int64_t>(ceil_div(warps, (int64_t)8), (int64_t)ctx->num_sms * 8));
    e = vec ? launch_early(orth_split_kernel<DT, true>, g, 256, 0, ctx->stream, a)
            : launch_early(orth_split_kernel<DT, false>, g, 256, 0, ctx->stream, a);
  }
  return e == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

// Scratch of the narrow kernel: norms and the barrier's counter, A, its parts.
int64_t small_bytes(int64_t s, int64_t l) {
  const int64_t s16 = round_up(s, 16), ctas = ceil_div(l, (int64_t)kSmallCols);
  return round_up(ctas * 8, 256) + 256 + (1 + ctas) * s16 * s16 * 4;
}

gc_status launch_small(gc_ctx* ctx, SmallArgs& a, char* at) {
  static uint64_t devices = 0;
  if (!allow_smem(ctx, orth_small_kernel, (int)kSmallSmem, devices)) return GC_ERR_CUDA;
  const int64_t ctas = ceil_div(a.l, (int64_t)kSmallCols);
  a.s16 = (int)round_up(a.s, 16);
  a.status = ctx->ws.status;
  a.norms = reinterpret_cast<double*>(at);
  at += round_up(ctas * 8, 256);
  a.arrived = reinterpret_cast<uint32_t*>(at);
  at += 256;
  a.gram = reinterpret_cast<uint32_t*>(at);
  at += (int64_t)a.s16 * a.s16 * 4;
  a.part = reinterpret_cast<float*>(at);
  if (ctas > 1 && cudaMemsetAsync(a.arrived, 0, 4, ctx->stream) != cudaSuccess) return GC_ERR_CUDA;
  LaunchScope L(ctx, GC_PHASE_ORTH_PRODUCT);
  void* args[] = {&a};
  const cudaError_t e =
      ctas > 1 ? cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(orth_small_kernel),
                                             dim3((unsigned)ctas), dim3(256), args, kSmallSmem,
                                             ctx->stream)
               : cudaLaunchKernel(reinterpret_cast<const void*>(orth_small_kernel), dim3(1),
                                  dim3(256), args, kSmallSmem, ctx->stream);
  return e == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

}  // namespace

int64_t orth_scratch_bytes(int64_t m, int64_t n) {
  if (m == 0 || n == 0) return 0;
  const int64_t s = std::min(m, n), l = std::max(m, n);
  int64_t bytes = kMaxParts * 8 + kTopBytes + round_up(kArrivedBytes, 256) + 2 * planes_bytes(s, l) +
                  2 * planes_bytes(s, s) + parts_bytes(s, l);
  if (s <= kSmallS) bytes = std::max(bytes, small_bytes(s, l));
  return bytes;
}

gc_status launch_orth(gc_ctx* ctx, const void* g, int dtype, int64_t m, int64_t n, int64_t ldg,
                      int steps, const float* coefs, float eps, float scale, void* out,
                      int odtype, int64_t ldo, void* scratch) {
  if (m == 0 || n == 0) return GC_OK;
  const int64_t s = std::min(m, n), l = std::max(m, n);
  char* at = static_cast<char*>(scratch);
  if (s <= kSmallS && ceil_div(l, (int64_t)kSmallCols) <= ctx->num_sms && steps <= kSmallSteps) {
    SmallArgs a{};
    a.g = g;
    a.out = out;
    a.l = l;
    a.ldg = ldg;
    a.ldo = ldo;
    a.s = (int)s;
    a.tall = m > n;
    a.dtype = dtype;
    a.odtype = odtype;
    a.steps = steps;
    a.eps = eps;
    a.scale = scale;
    for (int k = 0; k < 3 * steps; ++k) a.coefs[k / 3][k % 3] = coefs[k];
    return launch_small(ctx, a, at);
  }
  InputArgs in{};
  in.part = reinterpret_cast<double*>(at);
  at += kMaxParts * 8;
  in.top = reinterpret_cast<uint32_t*>(at);
  Range* const ranges = reinterpret_cast<Range*>(in.top + kMaxParts);
  in.range = ranges;
  at += kTopBytes;
  in.arrived = reinterpret_cast<uint32_t*>(at);
  at += round_up(kArrivedBytes, 256);
  auto planes = [&](int64_t rows, int64_t cols) {
    Planes p{reinterpret_cast<uint16_t*>(at), rows, cols, plane_pitch(cols), 0};
    p.size = rows * p.pitch;
    at += planes_bytes(rows, cols);
    return p;
  };
  Planes x = planes(s, l), next = planes(s, l);
  const Planes gram = planes(s, s), poly = planes(s, s);
  in.g = g;
  in.m = m;
  in.n = n;
  in.ld = ldg;
  in.pitch = x.pitch;
  in.plane_size = x.size;
  in.dst = x.at;
  in.eps = eps;
  in.parts = (int)std::min<int64_t>(ceil_div(m * ceil_div(n, (int64_t)256), (int64_t)8),
                                    std::min(kMaxParts, ctx->num_sms * 4));
  gc_status st = dtype == GC_F32    ? input<GC_F32>(ctx, in)
                 : dtype == GC_BF16 ? input<GC_BF16>(ctx, in)
                                    : input<GC_F16>(ctx, in);
  float* const part = reinterpret_cast<float*>(at);
  for (int k = 0; st == GC_OK && k < steps; ++k) {
    ProductArgs a{};
    a.part = part;
    a.arrived = in.arrived;
    const bool one = k == 0 && dtype != GC_F32;  // X is one plane
    a.range = ranges + (k & 1);
    a.next_range = ranges + (~k & 1);
    a.a_planes = a.b_planes = one ? 1 : 2;
    a.a = coefs[3 * k];
    a.b = coefs[3 * k + 1];
    a.c = coefs[3 * k + 2];
    st = product<kGram>(ctx, x, x, gram, a);
    if (st != GC_OK) break;
    a.prev = gram.at;
    a.a_planes = a.b_planes = 2;
    st = product<kPoly>(ctx, gram, gram, poly, a);
    if (st != GC_OK) break;
    a.b_planes = one ? 1 : 2;
    if (k + 1 < steps) {
      st = product<kApply>(ctx, poly, x, next, a);
      std::swap(x, next);
    } else {
      a.out = out;
      a.odtype = odtype;
      a.ldo = ldo;
      a.scale = scale;
      a.transposed = m > n;
      a.out_vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0 &&
                  (m == 1 || row_aligned(ldo, odtype));
      st = product<kLast>(ctx, poly, x, next, a);
    }
  }
  if (st != GC_OK) return st;
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

}  // namespace gc
