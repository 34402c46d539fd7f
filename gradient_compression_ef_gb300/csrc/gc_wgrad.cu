// gc_wgrad.cu -- the weight and bias gradients of a linear layer from the
// output's gradient and the 8-bit checkpoint of its input:
//
//   dw[o][i] (+)= sum over tokens t of dy[t][o] x^[t][i]
//   db[o]    (+)= sum over tokens t of dy[t][o]
//
// A matrix product whose sum runs over the rows of both operands, on the
// tensor cores (tcgen05, 16-bit operands, fp32 accumulation).  The first MMA
// operand is x^, the second dy, so that a thread's tensor-memory lane is an
// input column: 32 lanes store 32 consecutive floats of a row of dw, whatever
// its stride.  Both operands have the sum's axis as their slow one in memory;
// the descriptors say so (MN-major) and nothing is transposed.
//
// One persistent CTA pair per two SMs (cta_group::2) owns a tile of 256
// inputs x 256 outputs; each CTA holds 128 input columns of x^ and 128
// output columns of dy per block of 64 tokens.
//   producers two threads: TMA of dy (128-byte swizzle); of codes and scale bytes
//   db        one warp: column sums of dy, through a ring of boxes of its own
//   converter two groups of 4 warps, every second block each: codes -> bf16
//             (or fp16) operand in shared memory
//   issuer    one thread of the leader CTA: the MMAs of the pair
//   read-out  8 warps: tensor memory -> running sums in registers -> dw
//
// Bound by the tensor cores where there are tiles for every pair: 8192 x 4096
// -> 11008 bf16 with db takes 414 us, 1784 Tflop/s (cuBLAS reaches 1874 on this
// GPU in a burst), and 486 us, 1519, back to back for seconds, when the power
// limit lowers the clock (cuBLAS then 1728); fp16 478 us, 1546: its conversion
// takes an instruction more for every two values and holds the tensor cores up.  db costs 2 to 7 us of that; nobody
// waits for its warp, which takes about 0.5 us for a box of 64 x 64.  (By a
// kernel of its own before the product db cost 25 us, and a launch: 100 x 512
// -> 512 bf16 12.4 us, now 10.4.  Only where a layer has hardly any inputs is
// one warp too few: 8192 x 64 -> 11008 bf16 78 us by the kernel, 88 now.)
// Small products are latency: 32768 x 768 -> 512 fp16 34 us and the join; 2501
// x 1001 -> 2051 fp32 (three planes) 35 us beside the split, 17, and the join.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "gc_act8.cuh"
#include "gc_sm100.cuh"

namespace gc {
namespace {

constexpr int kTile = 256;           // inputs and outputs of a pair's tile
constexpr int kHalf = 128;           // of one CTA
constexpr int kTok = 64;             // tokens of a block
constexpr int kStages = 4;           // of operands
constexpr int kCodeStages = 6;       // of codes and scale bytes
constexpr uint32_t kOpBytes = kHalf * kTok * 2;     // one CTA's operand, 16 KB
constexpr uint32_t kCodeBytes = kHalf * kTok;       // 8 KB
constexpr uint32_t kScaleBytes = 16 * kTok;
constexpr int kReadWarps = 8, kConvWarps = 8;
constexpr int kGroups = 2, kGroupWarps = kConvWarps / kGroups;
// The groups take blocks in turn, so a stage is always the same group's.  It
// has to be: a group that met a stage's barrier at every other phase only
// could not tell by the parity which of the two it sees.
static_assert(kStages % kGroups == 0 && kCodeStages % kGroups == 0, "a stage has one group");
constexpr int kDyWarp = kReadWarps + kConvWarps, kIssuerWarp = kDyWarp + 1,
              kCodeWarp = kDyWarp + 2, kBiasWarp = kDyWarp + 3;
constexpr int kThreads = 640;        // 5 warpgroups
constexpr int kBiasStages = 4;       // boxes of 64 tokens x 64 outputs
constexpr uint32_t kBiasBytes = kTok * 64 * 2;
constexpr uint32_t kTmemCols = 512;  // two accumulators of 256 columns
constexpr int kSegBlocks = 8;        // token blocks per accumulator
constexpr int kMaxPairs = 96;
constexpr long long kWaitCycles = 4000000000ll;  // bound on each wait: ~2 s

// The work of a call: `tiles` output tiles of `blocks` token blocks.  Pair g
// takes whole tiles g, g + pairs, ... of the first `full`; the rest, too few
// for another round, are cut into ranges of `len` blocks of their joint
// (tile, block) sequence, one range per pair.
struct Plan {
  int64_t in_tiles, out_tiles, full, rest;
  int64_t blocks, tok_blocks;  // per tile (all planes); per plane
  int64_t len, ranges;
  int pairs;
};

struct WgradArgs {
  Plan plan;
  float *dw, *db;
  float* part;        // [2 * ranges][256 outputs][256 inputs]
  // db: bias_len token blocks of 64 outputs at a time are one of bias_items
  float* bias_part;    // [bias_parts][out], where there are several
  uint32_t bias_items;  // 0: no db asked for
  uint32_t bias_len, bias_parts, strips;
  uint32_t* status;
  int64_t out, in, lddw;
  int accumulate;
};

// One piece of a pair's work: blocks [k0, k1) of a tile; slot < 0: the whole
// tile, stored to dw.
struct Unit {
  int64_t tile, k0, k1, slot;
};

struct Work {
  const Plan& p;
  int64_t round, r0, r1;
  int g;
  __device__ __forceinline__ Work(const Plan& plan, int pair) : p(plan), round(0), g(pair) {
    r0 = min(p.len * g, p.rest * p.blocks);
    r1 = min(r0 + p.len, p.rest * p.blocks);
  }
  __device__ __forceinline__ bool next(Unit& u) {
    const int64_t t = round * p.pairs + g;
    if (t < p.full) {
      ++round;
      u = {t, 0, p.blocks, -1};
      return true;
    }
    if (r0 >= r1) return false;
    const int64_t tile = r0 / p.blocks, k0 = r0 - tile * p.blocks;
    const int64_t k1 = min(p.blocks, k0 + (r1 - r0));
    const int64_t first = p.len * g / p.blocks;  // the range's first tile
    u = {p.full + tile, k0, k1, (k0 == 0 && k1 == p.blocks) ? -1 : 2 * (int64_t)g + (tile - first)};
    r0 += k1 - k0;
    return true;
  }
};

// Tiles in bands of 8 input tiles, outputs fastest across a band: the tiles
// that pairs work on at the same time share their operand columns in L2.
__host__ __device__ inline void tile_place(const Plan& p, int64_t t, int64_t& it, int64_t& ot) {
  const int64_t per = 8 * p.out_tiles, band = t / per, r = t - band * per;
  const int64_t w = p.in_tiles - band * 8 < 8 ? p.in_tiles - band * 8 : 8;
  ot = r / w;
  it = band * 8 + r - ot * w;
}

struct Smem {
  uint32_t a, b, bias, codes, scales;  // shared addresses
  uint64_t *full, *empty, *cfull, *cempty, *acc_full, *acc_empty, *bfull, *drain;
  uint32_t* tmem_slot;
};

constexpr size_t kSmemBytes =
    1024 + (size_t)kStages * 2 * kOpBytes + (size_t)kBiasStages * kBiasBytes +
    (size_t)kCodeStages * (kCodeBytes + kScaleBytes) +
    8 * (2 * kStages + 2 * kCodeStages + kBiasStages + 5) + 16;

__device__ __forceinline__ Smem carve(unsigned char* base) {
  Smem s;
  const uint32_t at = (sm100::smem_u32(base) + 1023u) & ~1023u;
  unsigned char* p = base + (at - sm100::smem_u32(base));
  s.a = at;
  s.b = s.a + kStages * kOpBytes;
  s.bias = s.b + kStages * kOpBytes;
  s.codes = s.bias + kBiasStages * kBiasBytes;
  s.scales = s.codes + kCodeStages * kCodeBytes;
  uint64_t* bar = reinterpret_cast<uint64_t*>(p + (s.scales - at) + kCodeStages * kScaleBytes);
  s.full = bar;
  s.empty = s.full + kStages;
  s.cfull = s.empty + kStages;
  s.cempty = s.cfull + kCodeStages;
  s.acc_full = s.cempty + kCodeStages;
  s.acc_empty = s.acc_full + 2;
  s.bfull = s.acc_empty + 2;
  s.drain = s.bfull + kBiasStages;
  s.tmem_slot = reinterpret_cast<uint32_t*>(s.drain + 1);
  return s;
}

template <int N>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int by = 1) {
    st += by;
    if (st >= N) {
      st -= N;
      ph ^= 1u;
    }
  }
};

// A block's place in its plane of dy, counted up without divisions.
struct TokCursor {
  int32_t tb, per;
  __device__ __forceinline__ TokCursor(int64_t k, int64_t tok_blocks) : per((int32_t)tok_blocks) {
    tb = (int32_t)((uint32_t)k % (uint32_t)per);
  }
  __device__ __forceinline__ void next() {
    if (++tb == per) tb = 0;
  }
};

__device__ __forceinline__ void sts_u4(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// decode2 in fp16: +-(16 + m * 2^-6) less +-16 is +-m * 2^-6; times
// 2^(B - 128), a power of two that fp16 holds for every B an fp16 value can
// have (104 .. 143), subnormals included.  SEL: a code in the low byte of each
// half, its sign spread over the high byte.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t two_f16(uint32_t w, uint32_t scale) {
  uint32_t v, d;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(v) : "r"(w), "n"(SEL));
  const uint32_t x = (v & 0x807F807Fu) | 0x4C004C00u, c = (v & 0x80008000u) | 0x4C004C00u;
  asm("{\n\t.reg .b32 t;\n\tsub.rn.f16x2 t, %1, %2;\n\tmul.rn.f16x2 %0, t, %3;\n\t}"
      : "=r"(d)
      : "r"(x), "r"(c), "r"(scale));
  return d;
}

// 2^(B - 128) in both halves; 0 below fp16's range, NaN above it.
__device__ __forceinline__ uint32_t f16_scale(uint32_t b) {
  const float f = __uint_as_float((max(b, 1u) - 1u) << 23);
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(h) : "f"(f));
  return b > 143u ? 0x7E007E00u : h;
}

template <bool F16>
__device__ __forceinline__ uint4 eight(uint32_t w0, uint32_t w1, uint32_t s) {
  if (F16)
    return make_uint4(two_f16<0x9180>(w0, s), two_f16<0xB3A2>(w0, s), two_f16<0x9180>(w1, s),
                      two_f16<0xB3A2>(w1, s));
  return make_uint4(decode2(w0, 0x1100u, s), decode2(w0, 0x3322u, s), decode2(w1, 0x1100u, s),
                    decode2(w1, 0x3322u, s));
}

template <bool F16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap map_dy,
                 const __grid_constant__ CUtensorMap map_codes,
                 const __grid_constant__ CUtensorMap map_scales,
                 const __grid_constant__ WgradArgs a) {
  using namespace sm100;
  extern __shared__ unsigned char wg_smem[];
  const Smem s = carve(wg_smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 2 * kGroupWarps + 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < kCodeStages; ++i) {
      mbar_init(&s.cfull[i], 1);
      mbar_init(&s.cempty[i], kGroupWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], 2 * kReadWarps);
    }
    for (int i = 0; i < kBiasStages; ++i) mbar_init(&s.bfull[i], 1);
    mbar_init(s.drain, 1);
    mbar_fence_init();
  }
  if (warp == kIssuerWarp) {
    tmem_alloc_pair(s.tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // the pair's barriers exist before either CTA arrives on one
  tc_fence_after_sync();
  const uint32_t tmem = *s.tmem_slot;
  bool ok = true;
  Work work(a.plan, pair);
  Unit u;

  if (warp >= kDyWarp) {
    reg_dec<64>();
    // These three warps run their loops as whole warps (uniform registers);
    // one elected lane issues.
    if (warp == kCodeWarp) {
      Ring<kCodeStages> ring;
      uint32_t loads = 0;
      while (ok && work.next(u)) {
        int64_t it, ot;
        tile_place(a.plan, u.tile, it, ot);
        const int32_t x = (int32_t)(it * kTile) + (int32_t)rank * kHalf;
        const int32_t xs = x / kActGroup & ~15;
        TokCursor cur(u.k0, a.plan.tok_blocks);
        for (int32_t n = (int32_t)(u.k1 - u.k0); n > 0; --n, ring.next(), cur.next()) {
          const int st = ring.st;
          if (loads >= kCodeStages) {
            if (!mbar_wait(&s.cempty[st], ring.ph ^ 1u, kWaitCycles)) ok = false;
            if (__any_sync(0xffffffffu, !ok)) {
              ok = false;
              break;
            }
          } else {
            ++loads;
          }
          if (elect_one()) {
            // the converters read the stage through the generic proxy, TMA
            // refills it through the asynchronous one
            fence_proxy_async_smem();
            const int32_t y = cur.tb * kTok;
            mbar_arrive_expect_tx(&s.cfull[st], kCodeBytes + kScaleBytes);
            tma_load_2d(s.codes + st * kCodeBytes, &map_codes, x, y, &s.cfull[st]);
            tma_load_2d(s.scales + st * kScaleBytes, &map_scales, xs, y, &s.cfull[st]);
          }
        }
      }
    } else if (warp == kDyWarp) {
      const uint32_t bar0 = map_to_rank(smem_u32(s.full), 0);  // the leader counts the bytes
      after_previous();  // dy's planes
      Ring<kStages> ring;
      uint32_t loads = 0;
      while (ok && work.next(u)) {
        int64_t it, ot;
        tile_place(a.plan, u.tile, it, ot);
        const int32_t x = (int32_t)(ot * kTile) + (int32_t)rank * kHalf;
        int32_t y = (int32_t)u.k0 * kTok;  // planes follow one another without a gap
        for (int32_t n = (int32_t)(u.k1 - u.k0); n > 0; --n, ring.next(), y += kTok) {
          const int st = ring.st;
          if (loads >= kStages) {
            // free once the pair's MMAs read it
            if (!mbar_wait_cluster(&s.empty[st], ring.ph ^ 1u, kWaitCycles)) ok = false;
            if (__any_sync(0xffffffffu, !ok)) {
              ok = false;
              break;
            }
          } else {
            ++loads;
          }
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(&s.full[st], 2 * kOpBytes);
            const uint32_t dst = s.b + st * kOpBytes;
            tma_load_2d_pair(dst, &map_dy, x, y, bar0 + st * 8);
            tma_load_2d_pair(dst + kOpBytes / 2, &map_dy, x + 64, y, bar0 + st * 8);
          }
        }
      }
      // the arrivals of the last MMAs on this CTA's barriers: none may be
      // under way when the CTA ends
      for (int i = 0; ok && i < kStages; ++i, ring.next()) {
        if (loads < kStages && (uint32_t)ring.st >= loads) continue;  // never filled
        if (!mbar_wait_cluster(&s.empty[ring.st], ring.ph ^ 1u, kWaitCycles)) ok = false;
      }
    } else if (warp == kIssuerWarp && rank == 0) {
      constexpr uint32_t idesc = idesc_f16_mn(kTile, kTile, F16 ? 0 : 1);
      // MN-major operands: 128-byte rows of 64 columns, 8 tokens per
      // 1024-byte group, the two blocks of 64 columns 8 KB apart; 16 tokens
      // (one MMA) are 2048 bytes
      const uint64_t da = smem_desc_sw128(s.a, kOpBytes / 2, 1024);
      const uint64_t db = smem_desc_sw128(s.b, kOpBytes / 2, 1024);
      const uint32_t hi = (uint32_t)(da >> 32);
      const uint32_t a0 = (uint32_t)da, b0 = (uint32_t)db;
      Ring<kStages> ring;
      uint32_t seg = 0;
      while (ok && work.next(u)) {
        int in_seg = 0;
        for (int32_t n = (int32_t)(u.k1 - u.k0); n > 0; --n, ring.next()) {
          const int st = ring.st;
          const uint32_t buf = seg & 1u;
          if (in_seg == 0 && seg >= 2 &&
              !mbar_wait_cluster(&s.acc_empty[buf], ((seg >> 1) - 1u) & 1u, kWaitCycles))
            ok = false;
          if (ok && !mbar_wait_cluster(&s.full[st], ring.ph, kWaitCycles)) ok = false;
          if (__any_sync(0xffffffffu, !ok)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const bool last = in_seg == kSegBlocks - 1 || n == 1;
          if (elect_one()) {
            const uint32_t off = (uint32_t)st * (kOpBytes >> 4), d = tmem + buf * kTile;
#pragma unroll
            for (int kk = 0; kk < kTok / 16; ++kk)
              mma_f16_pair(d, a0 + off + kk * (2048 >> 4), b0 + off + kk * (2048 >> 4), hi, idesc,
                           (in_seg | kk) ? 1u : 0u);
            mma_commit_pair(&s.empty[st]);
            if (last) mma_commit_pair(&s.acc_full[buf]);
          }
          ++in_seg;
          if (last) {
            ++seg;
            in_seg = 0;
          }
        }
      }
    }
    // Column sums of dy, beside the product and out of its way: a box is added
    // up by itself (16 additions), then to the item's sum.
    if (warp == kBiasWarp && a.bias_items > 0) {
      after_previous();
      const int c = lane & 7, r = lane >> 3;  // 16-byte chunk, first row
      const uint32_t off0 = (uint32_t)(r * 128 + ((c ^ r) << 4));
      const uint32_t off1 = (uint32_t)(r * 128 + ((c ^ (r + 4)) << 4));
      // every gridDim.x-th item; box k .. k1 of `item` is the next to load,
      // `left` boxes of `use` are to be added up
      const uint32_t blocks = (uint32_t)a.plan.blocks;
      uint32_t item = blockIdx.x, use = item, k = 0, k1 = 0, left = 0, x = 0;
      int32_t y = 0;
      auto more = [&] { return k < k1 || item < a.bias_items; };
      auto load = [&](int st) {
        if (k >= k1) {
          const uint32_t part = item / a.strips;
          x = (item - part * a.strips) * 64;
          k = part * a.bias_len;
          k1 = min(blocks, k + a.bias_len);
          item += gridDim.x;
          y = (int32_t)(k * kTok);
        }
        if (elect_one()) {
          fence_proxy_async_smem();  // the warp read the stage through the generic proxy
          mbar_arrive_expect_tx(&s.bfull[st], kBiasBytes);
          tma_load_2d(s.bias + st * kBiasBytes, &map_dy, (int32_t)x, y, &s.bfull[st]);
        }
        ++k;
        y += kTok;
      };
      for (int i = 0; i < kBiasStages && more(); ++i) load(i);
      float2 sum[4] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
      Ring<kBiasStages> ring;
      for (; use < a.bias_items; ring.next()) {
        const uint32_t part = use / a.strips;
        if (left == 0) left = min(blocks - part * a.bias_len, a.bias_len);
        const bool got = mbar_wait(&s.bfull[ring.st], ring.ph, kWaitCycles);
        if (__any_sync(0xffffffffu, !got)) {
          ok = false;
          break;
        }
        const uint32_t at = s.bias + ring.st * kBiasBytes;
        float2 box[4] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
          uint4 raw[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) raw[e] = lds_u128(at + (e & 1 ? off1 : off0) + (i + e) * 512);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float2 v[4];
            unpack2<F16 ? GC_F16 : GC_BF16>(raw[e], v);
#pragma unroll
            for (int j = 0; j < 4; ++j) box[j] = __fadd2_rn(box[j], v[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = __fadd2_rn(sum[j], box[j]);
        __syncwarp();
        if (more()) load(ring.st);
        if (--left) continue;
        const int64_t o = (int64_t)(use - part * a.strips) * 64 + c * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float t = j & 1 ? sum[j / 2].y : sum[j / 2].x;
          t += __shfl_xor_sync(0xffffffffu, t, 8);
          t += __shfl_xor_sync(0xffffffffu, t, 16);
          if (r == 0 && o + j < a.out) {
            if (a.bias_parts > 1) a.bias_part[part * a.out + o + j] = t;
            else a.db[o + j] = a.accumulate ? a.db[o + j] + t : t;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = both(0.0f);
        use += gridDim.x;
      }
    }
    // MMAs still in flight read both CTAs' shared memory: wait for them (the
    // commit of the lane that issued them).  In each CTA it is the dy producer
    // that waits, having kept step with the MMAs as far as here: a warp that
    // had nothing else to do would wait for the whole kernel, and a kernel of
    // more than kWaitCycles would look like one that hangs.
    if (warp == kIssuerWarp && rank == 0 && elect_one()) mma_commit_pair(s.drain);
    if (warp == kDyWarp && !mbar_wait_cluster(s.drain, 0, kWaitCycles)) ok = false;
  } else if (warp >= kReadWarps) {
    reg_dec<48>();
    const int cw = warp - kReadWarps, group = cw / kGroupWarps;
    const int unit = lane & 7, row0 = (cw % kGroupWarps) * 16 + (lane >> 3);
    const uint32_t half = (uint32_t)(unit >> 2);
    const uint32_t full0 = map_to_rank(smem_u32(s.full), 0);
    Ring<kStages> ring;
    Ring<kCodeStages> cring;
    ring.next(group);
    cring.next(group);
    int64_t done = group, skip = group;  // block of this CTA, blocks to pass over
    while (ok && work.next(u)) {
      int64_t it, ot;
      tile_place(a.plan, u.tile, it, ot);
      const uint32_t sat =
          (uint32_t)(((it * kTile + rank * kHalf) / kActGroup & 15) + (unit >> 1));
      int64_t k = u.k0 + skip;
      for (; k < u.k1;
           k += kGroups, done += kGroups, ring.next(kGroups), cring.next(kGroups)) {
        const int st = ring.st, cs = cring.st;
        bool got = mbar_wait(&s.cfull[cs], cring.ph, kWaitCycles);
        if (got && done >= kStages) got = mbar_wait_cluster(&s.empty[st], ring.ph ^ 1u, kWaitCycles);
        if (__any_sync(0xffffffffu, !got)) {
          ok = false;
          break;
        }
        uint4 c[4];
        uint32_t b[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t r = (uint32_t)(row0 + p * 4);
          c[p] = lds_u128(s.codes + cs * kCodeBytes + r * kHalf + unit * 16);
          b[p] = lds_u8(s.scales + cs * kScaleBytes + r * 16 + sat);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t r = (uint32_t)(row0 + p * 4);
          const uint32_t sc = F16 ? f16_scale(b[p]) : b[p] * 0x00800080u;
          // the codes that are stored first and second: lower and upper
          // eight, in the upper half's threads the other way round
          const uint4 one = eight<F16>(half ? c[p].z : c[p].x, half ? c[p].w : c[p].y, sc);
          const uint4 two = eight<F16>(half ? c[p].x : c[p].z, half ? c[p].y : c[p].w, sc);
          // 16-byte chunks 2 (unit % 4) and + 1 of the half's 128-byte row r,
          // swizzled; the upper half's threads store theirs in the other
          // order, so that eight threads cover all banks at each store
          const uint32_t row = s.a + st * kOpBytes + half * (kOpBytes / 2) + r * 128;
          const uint32_t ch = (uint32_t)(unit & 3) * 2;
          const uint32_t first = ((ch + half) ^ (r & 7u)) << 4;
          sts_u4(row + first, one);
          sts_u4(row + (first ^ 16u), two);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s.cempty[cs]);
          mbar_arrive_cluster(full0 + st * 8);
        }
        __syncwarp();
      }
      skip = k - u.k1;
    }
  } else {
    reg_inc<160>();
    // warp w reads lanes 32 (w % 4) .. + 31 (inputs) of columns 128 (w / 4)
    // .. + 127 (outputs) of every accumulator
    const uint32_t q = (uint32_t)warp & 3u, ch = (uint32_t)warp >> 2;
    const uint32_t acc_empty0 = map_to_rank(smem_u32(s.acc_empty), 0);
    uint32_t seg = 0;
    while (ok && work.next(u)) {
      float sum[kHalf];
#pragma unroll
      for (int c = 0; c < kHalf; ++c) sum[c] = 0.0f;
      for (int64_t k = u.k0; k < u.k1; k += kSegBlocks, ++seg) {
        const uint32_t buf = seg & 1u;
        const bool got = mbar_wait_cluster(&s.acc_full[buf], (seg >> 1) & 1u, kWaitCycles);
        if (__any_sync(0xffffffffu, !got)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t at = tmem + ((q * 32) << 16) + buf * kTile + ch * kHalf;
#pragma unroll
        for (int j = 0; j < kHalf / 16; ++j) {
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
      int64_t it, ot;
      tile_place(a.plan, u.tile, it, ot);
      const uint32_t m = rank * kHalf + q * 32 + lane, n = ch * kHalf;
      if (u.slot >= 0) {
        float* dst = a.part + (u.slot * kTile + n) * kTile + m;
#pragma unroll
        for (int c = 0; c < kHalf; ++c) dst[c * kTile] = sum[c];
      } else {
        const int64_t i = it * kTile + m, o = ot * kTile + n;
        float* w = a.dw + o * a.lddw + i;
        const int rows = (int)min((int64_t)kHalf, a.out - o);
        if (i < a.in) {
          if (a.accumulate) {
#pragma unroll
            for (int c = 0; c < kHalf; ++c, w += a.lddw)
              if (c < rows) *w += sum[c];
          } else {
#pragma unroll
            for (int c = 0; c < kHalf; ++c, w += a.lddw)
              if (c < rows) *w = sum[c];
          }
        }
      }
    }
  }
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
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// Adds the ranges' partials of a cut tile in the order of their tokens and
// stores it (join_rows outputs of a rest tile per block), and the partial rows
// of db (32 columns per block; the first blocks).  A block's time is one trip
// to L2 per four outputs and four partials.
__global__ void __launch_bounds__(256) wgrad_join_kernel(const __grid_constant__ WgradArgs a,
                                                         int bias_blocks, int join_rows) {
  const Plan& p = a.plan;
  if ((int)blockIdx.x < bias_blocks) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t o = (int64_t)blockIdx.x * 32 + lane;
    after_previous();
    float v = 0.0f;
    if (o < a.out) {
#pragma unroll 8
      for (int i = warp; i < (int)a.bias_parts; i += 8) v += a.bias_part[i * a.out + o];
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && o < a.out) {
#pragma unroll
      for (int w = 1; w < 8; ++w) v += s[w][lane];
      a.db[o] = a.accumulate ? a.db[o] + v : v;
    }
    return;
  }
  const int64_t b = blockIdx.x - bias_blocks, t = b / (kTile / join_rows);
  const int n0 = (int)(b - t * (kTile / join_rows)) * join_rows;
  const int64_t b0 = t * p.blocks, b1 = b0 + p.blocks;
  const int64_t g0 = b0 / p.len, g1 = (b1 - 1) / p.len;
  int64_t it, ot;
  tile_place(p, p.full + t, it, ot);
  const int64_t i = it * kTile + threadIdx.x;
  // the tile is the second one of its first range if that range begins with
  // another tile, the first one of every other
  const int64_t second = t - p.len * g0 / p.blocks;
  after_previous();
  if (g0 == g1 || i >= a.in) return;  // one range held it all and stored it
  for (int n = n0; n < n0 + join_rows; n += 4) {
    const float* src = a.part + n * kTile + threadIdx.x;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t g = g0; g <= g1; g += 4) {
      float x[4][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t slot = 2 * (g + e) + (g + e == g0 ? second : 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[e][j] = g + e <= g1 ? src[slot * kTile * kTile + j * kTile] : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += x[e][j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t o = ot * kTile + n + j;
      if (o < a.out) {
        float* w = a.dw + o * a.lddw + i;
        *w = a.accumulate ? *w + v[j] : v[j];
      }
    }
  }
}

// dy as planes of 16-bit values with 16-byte rows that the tensor maps take:
// fp32 cut into three bf16 values whose sum it is (8 significant bits each,
// by truncation, so every remainder is exact and no plane overflows); 16-bit
// types as they are.  Rows past `rows` and columns past `out` are zero.  A
// warp takes 32 consecutive units of 16 bytes of one row of dy.
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(256) wgrad_split_kernel(const char* dy, const char* end,
                                                          int64_t rows, int64_t row_bytes,
                                                          int64_t dy_pitch, uint16_t* planes,
                                                          int64_t plane_rows, int64_t pitch) {
  using E = Elem<DT>;
  constexpr int V = E::V;
  let_next_begin();
  const int64_t segs = (pitch + 32 * V - 1) / (32 * V), total = plane_rows * segs;
  for (int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); at < total;
       at += (int64_t)gridDim.x * 8) {
    const int64_t r = at / segs, u = (at - r * segs) * 32 + (threadIdx.x & 31);
    const uint4 raw = r < rows ? load_unit<DT, ALIGNED>(dy + r * dy_pitch, u * 16, row_bytes, end)
                               : make_uint4(0u, 0u, 0u, 0u);
    if (u * V >= pitch) continue;
    uint16_t* dst = planes + r * pitch + u * V;
    if (DT == GC_F32) {
      uint32_t rest[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = rest[e] & 0xFFFF0000u;
          rest[e] = __float_as_uint(__fsub_rn(__uint_as_float(rest[e]), __uint_as_float(p[e])));
        }
        *reinterpret_cast<uint2*>(dst + k * plane_rows * pitch) =
            make_uint2(__byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
      }
    } else {
      *reinterpret_cast<uint4*>(dst) = raw;
    }
  }
}

// --- host ----------------------------------------------------------------------------------------

int plane_count(int dtype) { return dtype == GC_F32 ? 3 : 1; }

Plan make_plan(int64_t rows, int64_t out, int64_t in, int planes, int pairs) {
  Plan p;
  p.in_tiles = ceil_div(in, kTile);
  p.out_tiles = ceil_div(out, kTile);
  p.tok_blocks = ceil_div(rows, kTok);
  p.blocks = p.tok_blocks * planes;
  p.pairs = std::min(pairs, kMaxPairs);
  const int64_t tiles = p.in_tiles * p.out_tiles;
  p.full = tiles / p.pairs * p.pairs;
  p.rest = tiles - p.full;
  // the rest over all pairs; a range shorter than an accumulator's blocks
  // would cost more to join than it saves
  p.len = std::max(ceil_div(p.rest * p.blocks, (int64_t)p.pairs),
                   std::min<int64_t>(p.blocks, kSegBlocks));
  p.ranges = p.rest ? ceil_div(p.rest * p.blocks, p.len) : 0;
  return p;
}

int64_t up256(int64_t b) { return (b + 255) / 256 * 256; }

int64_t planes_bytes(int64_t rows, int64_t out, int dtype) {
  return up256((int64_t)plane_count(dtype) * round_up(rows, kTok) * round_up(out, 8) * 2);
}
constexpr int64_t kSlotBytes = (int64_t)kTile * kTile * 4;

// Token blocks of one partial row of db: 8 (512 tokens), more where the
// partial rows would be over kMaxBiasParts.
constexpr int kMaxBiasParts = 127;
int64_t bias_len(int64_t blocks) {
  return std::max<int64_t>(kSegBlocks, ceil_div(blocks, (int64_t)kMaxBiasParts));
}
int64_t bias_bytes(int64_t blocks, int64_t out) {
  const int64_t parts = ceil_div(blocks, bias_len(blocks));
  return parts > 1 ? up256(parts * out * 4) : 0;
}

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

// rows x cols elements of `size` bytes, rows `pitch` bytes apart, read in
// boxes of kTok rows x box columns; what lies outside reads as zero.
bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t rows,
              int64_t cols, int64_t pitch, uint32_t box, bool swizzle) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)pitch};
  const cuuint32_t boxes[2] = {box, (cuuint32_t)kTok};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, type, 2, const_cast<void*>(base), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DT>
void launch_split(gc_ctx* ctx, const void* dy, int64_t rows, int64_t out, int64_t lddy,
                       uint16_t* planes, int64_t plane_rows, int64_t pitch) {
  constexpr int kSize = elem_size(DT);
  const int64_t total = plane_rows * ceil_div(pitch, 32 * Elem<DT>::V);
  const unsigned g = (unsigned)std::min<int64_t>(ceil_div(total, 8), (int64_t)ctx->num_sms * 8);
  const char* p = static_cast<const char*>(dy);
  const char* end = p + ((rows - 1) * lddy + out) * kSize;
  const auto kernel =
      row_aligned(lddy, DT) ? wgrad_split_kernel<DT, true> : wgrad_split_kernel<DT, false>;
  LaunchScope L(ctx, GC_PHASE_WGRAD_SPLIT);
  kernel<<<g, 256, 0, ctx->stream>>>(p, end, rows, out * kSize, lddy * kSize, planes, plane_rows,
                                     pitch);
}

template <bool F16>
gc_status launch_tiles(gc_ctx* ctx, const CUtensorMap& md, const CUtensorMap& mc,
                       const CUtensorMap& ms, const WgradArgs& a, bool early) {
  static uint64_t devices = 0;
  if (!allow_smem(ctx, wgrad_kernel<F16>, (int)kSmemBytes, devices)) return GC_ERR_CUDA;
  const int64_t pairs =
      a.plan.full ? a.plan.pairs
                  : std::min<int64_t>(a.plan.pairs,
                                      std::max(a.plan.ranges, ceil_div((int64_t)a.bias_items, 2)));
  LaunchScope L(ctx, GC_PHASE_WGRAD);
  if (early)
    return launch_early(wgrad_kernel<F16>, dim3((unsigned)(2 * pairs)), kThreads, kSmemBytes,
                        ctx->stream, md, mc, ms, a) == cudaSuccess
               ? GC_OK
               : GC_ERR_CUDA;
  wgrad_kernel<F16><<<(unsigned)(2 * pairs), kThreads, kSmemBytes, ctx->stream>>>(md, mc, ms, a);
  return GC_OK;
}

// The tiles and db, with dy's planes where they are needed.
gc_status launch_product(gc_ctx* ctx, const void* dy, int dtype, int64_t lddy,
                         const uint8_t* codes, const uint8_t* scales, int64_t rows,
                         uint16_t* planes, const WgradArgs& a) {
  const int64_t out = a.out, in = a.in;
  // the tensor map takes dy as it lies when its rows start on 16-byte
  // boundaries
  const void* d16 = dy;
  int64_t d_rows = rows, d_cols = out, d_pitch = lddy * 2;
  const bool split = dtype == GC_F32 || (rows > 1 && lddy * 2 % 16 != 0);
  if (split) {
    d_cols = round_up(out, 8);
    d_pitch = d_cols * 2;
    d_rows = a.plan.blocks * kTok;
    d16 = planes;
    if (dtype == GC_F32)
      launch_split<GC_F32>(ctx, dy, rows, out, lddy, planes, a.plan.tok_blocks * kTok, d_cols);
    else launch_split<GC_BF16>(ctx, dy, rows, out, lddy, planes, a.plan.tok_blocks * kTok, d_cols);
  } else if (rows == 1) {
    d_pitch = round_up(out * 2, 16);
  }
  const bool f16 = dtype == GC_F16;
  CUtensorMap md, mc, ms;
  const int64_t cp = ckpt_codes_pitch(in), sp = ckpt_scales_pitch(in);
  if (!make_map(&md, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d16,
                d_rows, d_cols, d_pitch, 64, true))
    return GC_ERR_CUDA;
  mc = ms = md;  // without inputs there are no tiles to read codes for
  if (in && (!make_map(&mc, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, rows, cp, cp, kHalf, false) ||
             !make_map(&ms, CU_TENSOR_MAP_DATA_TYPE_UINT8, scales, rows, sp, sp, 16, false)))
    return GC_ERR_CUDA;
  // behind the split the kernel may begin early: only dy waits for the planes
  return f16 ? launch_tiles<true>(ctx, md, mc, ms, a, split)
             : launch_tiles<false>(ctx, md, mc, ms, a, split);
}

}  // namespace

int64_t wgrad_scratch_bytes(int64_t rows, int64_t out, int64_t in, int dtype) {
  if (rows == 0 || out == 0) return 0;
  // partials of at most two slots per range, never more than one range per
  // pair; a plane of 16-bit dy in case its rows are not 16-byte aligned
  const Plan p = make_plan(rows, out, in, plane_count(dtype), kMaxPairs);
  const int64_t tiles = p.in_tiles * p.out_tiles;
  const int64_t slots = std::min<int64_t>(2 * kMaxPairs, tiles * p.blocks);
  return planes_bytes(rows, out, dtype) + slots * kSlotBytes + bias_bytes(p.blocks, out);
}

gc_status launch_wgrad(gc_ctx* ctx, const void* dy, int dtype, int64_t lddy, const uint8_t* codes,
                       const uint8_t* scales, int64_t rows, int64_t out, int64_t in, float* dw,
                       int64_t lddw, float* db, int accumulate, void* scratch) {
  if (out == 0) return GC_OK;
  if (rows == 0) {
    if (accumulate) return GC_OK;
    if ((in && cudaMemset2DAsync(dw, lddw * 4, 0, in * 4, out, ctx->stream) != cudaSuccess) ||
        (db && cudaMemsetAsync(db, 0, out * 4, ctx->stream) != cudaSuccess))
      return GC_ERR_CUDA;
    return GC_OK;
  }
  if (in == 0 && !db) return GC_OK;
  WgradArgs a{};
  a.plan = make_plan(rows, out, in, plane_count(dtype), ctx->num_sms / 2);
  char* at = static_cast<char*>(scratch);
  a.bias_part = reinterpret_cast<float*>(at);
  at += bias_bytes(a.plan.blocks, out);
  uint16_t* planes = reinterpret_cast<uint16_t*>(at);
  at += planes_bytes(rows, out, dtype);
  a.part = reinterpret_cast<float*>(at);
  a.dw = dw;
  a.db = db;
  a.status = ctx->ws.status;
  a.out = out;
  a.in = in;
  a.lddw = lddw;
  a.accumulate = accumulate;
  if (db) {
    a.strips = (uint32_t)ceil_div(out, 64);
    a.bias_len = (uint32_t)bias_len(a.plan.blocks);
    a.bias_parts = (uint32_t)ceil_div(a.plan.blocks, a.bias_len);
    a.bias_items = a.bias_parts * a.strips;  // at most 2^7 parts, 2^24 strips
  }
  const gc_status st = launch_product(ctx, dy, dtype, lddy, codes, scales, rows, planes, a);
  if (st != GC_OK) return st;
  // Tiles in many parts are few, and have blocks of fewer outputs.  The whole
  // call by blocks of 4 and of 16, bf16, 76 ranges: 2048 tokens 15.0 and 16.7
  // us for 6 tiles, 18.7 and 18.6 for 16, 24.7 and 24.7 for 20, 24.8 and 22.8
  // for 24, 39.0 and 33.6 for 64; 16384 tokens 29.0 and 34.9, 39.5 and 39.9,
  // 45.4 and 45.8, 48.7 and 48.6, 114.6 and 110.5.
  const int join_rows = a.plan.ranges >= 4 * a.plan.rest ? 4 : 16;
  const int64_t tile_blocks =
      a.plan.ranges > a.plan.rest ? a.plan.rest * (kTile / join_rows) : 0;
  const int64_t bias_blocks = a.bias_parts > 1 ? ceil_div(out, 32) : 0;
  if (tile_blocks + bias_blocks > 0) {
    LaunchScope L(ctx, GC_PHASE_WGRAD_JOIN);
    if (launch_early(wgrad_join_kernel, dim3((unsigned)(tile_blocks + bias_blocks)), 256, 0,
                     ctx->stream, a, (int)bias_blocks, join_rows) != cudaSuccess)
      return GC_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

}  // namespace gc
