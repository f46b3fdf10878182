// Matrix products grouped by expert: the rows of each expert with its weights on
// the tensor cores, and the weights' gradients.
//
// One kernel computes transposed tiles D[m, n] = sum_k A[m, k] B[n, k], m an output
// feature (a TMEM lane) and n a row of the expert:
//
//   product            m: features of W[e]      n: rows of xs     k: width of xs
//   its dxs            m: width of W[e]         n: rows of dys    k: features
//   its dweight        m: outer index of dW[e]  n: its inner one  k: rows of the expert
//
// With the rows as the MMA's N, which may be any multiple of 16 (of 32 for a pair of blocks),
// an expert of few rows costs few columns and not a whole tile of 128.  fp32 accumulation in
// TMEM, of a long k in parts (kPartK), and one rounding at the store.  The products' tiles are
// turned over in shared memory on their way out; dweight's leave as they are, in boxes by the
// tensor memory accelerator.
//
// Blocks are resident: one warp fills a ring of 64-wide slices of A and B, one issues the MMAs,
// others store a tile while the next is computed.  What bounds it, measured on one GB300
// (L2 gives the multiprocessors at most about 15 TB/s together):
//   many rows   16384 rows 5120 -> 5120 bf16: 467 to 483 us, 1840 to 1780 TFLOP/s; the MMAs alone
//               386 us, the copies alone 467 us
//   some        128 experts of 256 rows 2048 -> 5120: 488 us; the weights' bytes at 6.8 TB/s: 396
//   one         128 experts of one row: 382 us, 7.0 TB/s
//   dweight     16384 rows 5120 x 5120: 496 to 524 us; 32 experts of 512 rows 5120 x 4096: 515 us,
//               where the stores meet the copies in L2; 128 experts of one row: 385 us, 7.0 TB/s
//   plain loads 61 experts of 72 rows 1023 -> 1001 fp16: 82 to 87 us, bound by the instructions
//               that shift rows into place
#pragma once

#include <cuda.h>

#include <atomic>

#include "hcmix_common.cuh"
#include "hcmix_gate.cuh"
#include "hcmix_sm100.cuh"
#include "hcmix_vec.cuh"

namespace hcmix {
namespace sublayer {

constexpr int kProductExperts = 4096;
constexpr int kTileM = 128, kTileK = 64;  // kTileM: of one block
constexpr int kBoxBytes = 64 * 128;               // 64 rows of 64 16-bit elements
enum class ProductMode { kRowsK, kRowsM, kWeight };  // A's contiguous index: k, m; dweight

// kCtas, the blocks that work together:
//   1  operands whose rows do not all start on 16 bytes, by plain loads and tiles of 128 x 128;
//   2  a pair: tcgen05 cta_group::2 with 256 features, and half of B in each block, so that
//      a multiprocessor's shared memory takes in and gives out two thirds of what a tile of
//      128 x 256 would need.
// No copy is sent to several blocks: operands may lie in a peer's memory.
constexpr int kABytes = kTileM * kTileK * 2;
__host__ __device__ constexpr int kTileN(int ctas) { return ctas > 1 ? 256 : 128; }
constexpr int kAccumulator = 256;  // TMEM columns
__host__ __device__ constexpr int kStageBytes(int ctas) {
  return kABytes + kTileN(ctas) * kTileK * 2 / ctas;
}
__host__ __device__ constexpr int kStages(int ctas) { return ctas > 1 ? 6 : 2; }
constexpr int kMostStages = 6;
// Row tiles of a panel, whose rows are read again for each of the features' tiles: few enough to
// stay in L2 beside the weights (128 experts of 256 rows 2048 -> 5120: panels of 5 MB 474 us, 10 MB
// 488, 20 MB 522, 40 MB 592; of like rows on average, but skewed, 685, 665, 682, 659; 32 experts
// of 256 to 767 rows 5120 -> 4096: 585, 585, 571, 558).
constexpr int64_t kPanelBytes = 10 << 20;
inline int panel_tiles(int64_t K) {
  const int64_t n = kPanelBytes / (kTileN(2) * K * 2);
  return (int)(n < 4 ? 4 : n > 64 ? 64 : n);
}
// The MMAs' sums drop what lies below the last place of the running sum at each step of 16 k,
// always towards zero, which adds up where roundings would average out (of 131072 rows: 1.5e-4 of
// a sum of random terms, 7.9e-4 of positive ones).  So a tile of a long k is computed in parts,
// each from zero, that the storing warps add up in fp32.  Parts of 16384 for a result of a 16-bit
// type drop at most 7.9e-5, a sixth of fp16's half step.  Parts of 1024 for an fp32 result leave
// 1.0e-6 (2.1e-6 of positive terms) at any length, a sum of 16384 fp32 roundings 1.5e-6 (1.9e-6).
// 16384 rows 5120 x 5120 fp32: parts of 1024 548 us, of 2048 526 (2.1e-6, 5.3e-6), in one go 511
// (1.9e-5, 7.9e-5).
constexpr int kPartK = 16384, kPartK32 = 1024;
constexpr int64_t kProductWait = 4000000000ll;  // cycles without a stage: about two seconds

// One operand as it lies in memory: rows of contiguous elements.
struct Matrix3 {
  const void* p;
  int64_t row, expert;  // strides in elements
  int inner, outer;     // extents; rows of experts: outer is set by each tile
};

struct ProductArgs {
  CUtensorMap a_map, b_map, b16_map;  // boxes of 64 x 64, and of 64 x 16
  CUtensorMap out_map;                // dweight: boxes of 32 rows of 128 bytes
  Matrix3 a, b;
  const int32_t* offsets;
  int64_t R;
  int E;
  int M, N, K;        // extents of m, n and k; product: N unused, dweight: K unused
  int panel;          // product: row tiles that take turns at the same features
  int part;           // k that are summed in one go, a multiple of 64
  int gated;          // A's rows M .. 2 M - 1 are u's features, those before g's
  void* out;          // product: [R, M]; dweight: [E, M, N]
  void* saved;        // gated: [R, 2 M] or null
  int f16, out_f32;
  int vec;            // rows of out (and saved) start on 16 bytes
};

// Set by a wait that was given up, on the device that it happened on.
static __device__ uint32_t g_product_error;

// A tile, or a part of one along k, as the scheduling warp tells the others.
struct alignas(16) ProductTile {
  int expert;
  int m0, m1;  // origins of the two halves (64 lanes each) of the block's A
  int n;       // valid rows of B; 0: no more tiles
  int n0;      // the first, or the first outer feature
  int k0;      // the first k; dweight: the expert's first row
  int depth;   // of k
  int part;    // kFirstPart, kLastPart or both
};
constexpr int kFirstPart = 1, kLastPart = 2;

// Plain loads.  A warp copies 16 rows of 64 elements as the aligned 16-byte blocks that hold
// them (at the matrix's two ends element by element) into a ring of its own, and when they
// have come, shifts them into their places in the swizzled stage.
constexpr int kRawRows = 16, kProducers = 256 / kRawRows;  // warps: a stage has 256 rows
constexpr int kRawDepth = 3, kRawPitch = 144, kRawBox = kRawRows * kRawPitch;
__host__ __device__ constexpr int kRawBytes(int ctas) {
  return ctas > 1 ? 0 : kProducers * kRawDepth * kRawBox;
}
struct RawRows {
  const char* at;  // the first row's first element
  int64_t pitch;   // bytes
  int elements;    // of a row; the others are zeros
  int rows;        // that there are; the others are zeros
};

constexpr int kQueue = 4;  // tiles told ahead
struct ProductControl {
  ProductTile tile[kQueue];
  uint64_t told[kQueue], taken[kQueue];
  uint64_t full[kMostStages], empty[kMostStages];
  // dweight by pairs: a block's last stage of a tile, and both blocks' zeroed ones
  uint64_t tail[kMostStages], ready[kMostStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  uint32_t copied;  // stages that the block's (first) copying warp has done with
  int64_t scan[32];
  RawRows raw[kProducers][kRawDepth];
};
// Warps that store: one or two for each 32 lanes of TMEM.
__host__ __device__ constexpr int kStorers(int ctas) { return ctas > 1 ? 8 : 4; }
// A storing warp's shared memory: half a chunk of 32 x 32 in fp32 or a rounded one; dweight: a
// box of 32 rows of 128 bytes.
__host__ __device__ constexpr int kTurnBytes(ProductMode mode) {
  return mode == ProductMode::kWeight ? 4096 : 2048;
}
// Shared memory of a block; dweight needs no table of the experts' tiles.
template <int kCtas, ProductMode kMode>
constexpr size_t product_smem(int E) {
  return 1024 + (size_t)kStages(kCtas) * kStageBytes(kCtas) +
         kStorers(kCtas) * kTurnBytes(kMode) + kRawBytes(kCtas) + sizeof(ProductControl) +
         (kMode == ProductMode::kWeight ? 0 : ((size_t)E + 1) * 4);
}
static_assert(product_smem<2, ProductMode::kRowsK>(kProductExperts) <= 227 * 1024 &&
                  product_smem<1, ProductMode::kRowsK>(kProductExperts) <= 227 * 1024 &&
                  product_smem<1, ProductMode::kWeight>(kProductExperts) <= 227 * 1024 &&
                  product_smem<2, ProductMode::kWeight>(kProductExperts) <= 227 * 1024,
              "shared memory of a block");

__device__ __forceinline__ int clamp_offset(int v, int64_t R) {
  return v < 0 ? 0 : v > R ? (int)R : v;
}
// The expert's rows, within 0 .. R whatever offsets holds.
__device__ __forceinline__ void expert_rows(const ProductArgs& A, int e, int& first, int& count) {
  first = clamp_offset(A.offsets[e], A.R);
  const int last = clamp_offset(A.offsets[e + 1], A.R);
  count = last > first ? last - first : 0;
}

// The number of row tiles of all experts before each, in `cum`, at most 2^31 - 1 (which only
// offsets that fall can pass: they may count rows many times over).
template <int kCtas>
__device__ __forceinline__ void count_tiles(const ProductArgs& A, int* cum, int64_t* scan) {
  const int threads = blockDim.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int per = (A.E + threads - 1) / threads;
  const int e0 = tid * per < A.E ? tid * per : A.E, e1 = e0 + per < A.E ? e0 + per : A.E;
  int64_t sum = 0;
  for (int e = e0; e < e1; ++e) {
    int first, count;
    expert_rows(A, e, first, count);
    const int tiles = (count + kTileN(kCtas) - 1) / kTileN(kCtas);
    cum[e + 1] = tiles;
    sum += tiles;
  }
  int64_t before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += t;
  }
  if (lane == 31) scan[warp] = before;
  __syncthreads();
  before -= sum;
  for (int w = 0; w < warp; ++w) before += scan[w];
  if (tid == 0) cum[0] = 0;
  for (int e = e0; e < e1; ++e) {
    before += cum[e + 1];
    cum[e + 1] = before < 0x7fffffff ? (int)before : 0x7fffffff;
  }
  __syncthreads();
}

// The MMA's N: a multiple of 16 for each block.
template <int kCtas>
__device__ __forceinline__ int round_rows(int n) {
  constexpr int to = 16 * kCtas;
  return (n + to - 1) / to * to;
}

// Features of a tile.
template <int kCtas>
__host__ __device__ __forceinline__ int tile_width(const ProductArgs& A) {
  return (A.gated ? kTileM / 2 : kTileM) * kCtas;
}

template <int kCtas, ProductMode kMode>
__device__ __forceinline__ int64_t tile_count(const ProductArgs& A, const int* cum) {
  const int width = tile_width<kCtas>(A);
  const int64_t mt = (A.M + width - 1) / width;
  if (kMode == ProductMode::kWeight) return A.E * mt * ((A.N + kTileN(kCtas) - 1) / kTileN(kCtas));
  return cum[A.E] * mt;
}

// Tile t, with the features of block `rank`.
template <int kCtas, ProductMode kMode>
__device__ __forceinline__ ProductTile tile_at(const ProductArgs& A, const int* cum, int64_t t,
                                               int rank) {
  ProductTile T = {};
  const int width = tile_width<kCtas>(A);
  const int64_t mt = (A.M + width - 1) / width;
  int64_t m;
  int first, count;
  if (kMode == ProductMode::kWeight) {
    const int64_t nt = (A.N + kTileN(kCtas) - 1) / kTileN(kCtas);
    T.expert = (int)(t / (mt * nt));
    const int64_t rest = t - T.expert * (mt * nt);
    m = rest / nt;
    T.n0 = (int)(rest - m * nt) * kTileN(kCtas);
    T.n = A.N - T.n0 < kTileN(kCtas) ? A.N - T.n0 : kTileN(kCtas);
    expert_rows(A, T.expert, first, count);
    T.k0 = first, T.depth = count;
  } else {
    // a panel's row tiles take turns at each of the features' tiles
    const int64_t panel = t / (A.panel * mt), rest = t - panel * (A.panel * mt);
    const int64_t q0 = panel * A.panel;
    const int64_t pn = cum[A.E] - q0 < A.panel ? cum[A.E] - q0 : A.panel;
    m = rest / pn;
    const int q = (int)(q0 + rest - m * pn);
    int lo = 0, hi = A.E;  // cum[lo] <= q < cum[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (cum[mid] <= q) lo = mid; else hi = mid;
    }
    T.expert = lo;
    expert_rows(A, lo, first, count);
    const int nt = cum[lo + 1] - cum[lo], j = q - cum[lo];
    // the expert's tiles are of like size, as far as the MMA's multiples allow: 300 rows are 160 and
    // 140, 513 are 192, 192 and 129, but 2049 still eight tiles of 256 and one of a row
    const int size = round_rows<kCtas>((count + nt - 1) / nt);
    T.n0 = first + j * size;
    T.n = count - j * size < size ? count - j * size : size;
    if (T.n > kTileN(kCtas)) T.n = kTileN(kCtas);  // (see count_tiles)
    T.depth = A.K;
  }
  T.m0 = (int)m * width + rank * (width / kCtas);
  T.m1 = A.gated ? A.M + T.m0 : T.m0 + kTileM / 2;
  T.part = kFirstPart | kLastPart;
  return T;
}

// dweight by pairs: an expert's last 64 rows, if they are fewer, are zeroed behind before they
// are multiplied, which takes about 2 us from their arrival.  So they are copied up to
// kTailLead stages early and still multiplied last.  Their place among the tile's stages; the
// number of stages where there are none such.  (32 experts of 256 to 767 rows 5120 x 4096: 602 us
// in their turn, 580 three stages early.)
constexpr int kTailLead = 3;
__device__ __forceinline__ int tail_place(int depth) {
  const int blocks = (depth + kTileK - 1) / kTileK;
  if (depth % kTileK == 0) return blocks;
  return blocks - 1 < kTailLead ? 0 : blocks - 1 - kTailLead;
}

// ---- plain loads, of matrices whose rows do not all start on 16 bytes.

__device__ __forceinline__ const char* align16(const char* p) {
  return reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15);
}

// The careful copy: no byte outside of low .. high - 1 is read, rows and elements that are not
// there are zeros.  
__device__ __forceinline__ void copy_raw(uint32_t raw, const RawRows& X, const char* low,
                                         const char* high, int lane) {
#pragma unroll 1
  for (int i = 0; i * 32 < kRawRows * 9; ++i) {  // nine blocks hold 128 bytes of any alignment
    const int at = i * 32 + lane, row = at / 9, block = at - 9 * row;
    if (kRawRows * 9 % 32 != 0 && row >= kRawRows) break;
    const char* from = X.at + row * X.pitch;
    const char* p = align16(from) + 16 * block;
    const uint32_t to = raw + row * kRawPitch + 16 * block;
    if (row < X.rows && p < from + 2 * X.elements && p + 16 > from) {
      if (p >= low && p + 16 <= high) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
      } else {
        for (int k = 0; k < 16; k += 2) {
          uint16_t v = 0;
          if (p + k >= low && p + k < high) v = *reinterpret_cast<const uint16_t*>(p + k);
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + k), "h"(v) : "memory");
        }
      }
    } else {
      sm100::sts128(to, make_uint4(0, 0, 0, 0));
    }
  }
}

// `dst`: the place of the first row, whose number in its box is a multiple of 8.
__device__ __forceinline__ void place_raw(uint32_t dst, uint32_t raw, const RawRows& X, int lane) {
  const int c = lane % 8;
  const uint32_t at = (uint32_t)reinterpret_cast<uintptr_t>(X.at), pitch = (uint32_t)X.pitch;
  const bool whole = X.elements >= kTileK;
#pragma unroll
  for (int i = 0; i < kRawRows / 4; ++i) {
    const int row = 4 * i + lane / 8;
    const uint32_t shift = at + row * pitch;  // its lower four bits
    const uint32_t from = raw + row * kRawPitch + 16 * c + (shift & 12);
    uint32_t w[5];
#pragma unroll
    for (int k = 0; k < 5; ++k)
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[k]) : "r"(from + 4 * k) : "memory");
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 8 * (shift & 2));
    if (!whole) {  // what lies behind a row's end is the next one's
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int left = X.elements - 8 * c - 2 * k;
        w[k] = left <= 0 ? 0 : left == 1 ? w[k] & 0xffffu : w[k];
      }
    }
    sm100::sts128(dst + row * 128 + ((c ^ (row & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
  }
}

// ---- descriptors.  K-major operands: smem_desc_sw128.  An operand whose rows are k and
// whose contiguous index is m (or n) lies in boxes of 64 of them: 8 k are 1024 bytes on,
// the next 64 m a box on.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(kBoxBytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// By a whole converged warp, issued by the lane that elect.sync picks (a branch on the lane
// would keep the descriptors out of uniform registers): MMAs of 16 k, and of the 64 of a stage,
// whose descriptors step by kA and kB.
template <bool kTma>
__device__ __forceinline__ void mma_16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  if constexpr (kTma)
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
template <bool kTma, int kA, int kB>
__device__ __forceinline__ void mma_64(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  if constexpr (kTma)
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t"
        ".reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 q, %4, %4;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "add.u64 a, %1, %5;\n\tadd.u64 b, %2, %6;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.u64 a, %1, %7;\n\tadd.u64 b, %2, %8;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.u64 a, %1, %9;\n\tadd.u64 b, %2, %10;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, q;}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "n"(kA), "n"(kB), "n"(2 * kA),
        "n"(2 * kB), "n"(3 * kA), "n"(3 * kB)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t"
        ".reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 q, %4, %4;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "add.u64 a, %1, %5;\n\tadd.u64 b, %2, %6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.u64 a, %1, %7;\n\tadd.u64 b, %2, %8;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.u64 a, %1, %9;\n\tadd.u64 b, %2, %10;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "n"(kA), "n"(kB), "n"(2 * kA),
        "n"(2 * kB), "n"(3 * kA), "n"(3 * kB)
        : "memory");
}
// An arrival at `bar`, in the blocks of `mask`, when the elected lane's MMAs so far are done.
template <bool kTma>
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t mask) {
  if constexpr (kTma)
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
        ".multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"((uint16_t)mask)
        : "memory");
  else
    sm100::umma_commit_warp(bar);
}

template <bool kTma>
__device__ __forceinline__ void product_tmem_alloc(uint32_t dst) {
  if constexpr (kTma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(dst)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    sm100::tmem_alloc(dst, 512);
    sm100::tmem_relinquish();
  }
}
template <bool kTma>
__device__ __forceinline__ void product_tmem_dealloc(uint32_t tmem) {
  if constexpr (kTma)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  else
    sm100::tmem_dealloc(tmem, 512);
}

// The address, in the cluster's shared memory, of what the pair's first block has at `addr`.
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
// One arrival at a barrier of that block.
template <bool kTma>
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
  if constexpr (kTma)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_leader(bar))
                 : "memory");
  else
    sm100::mbar_arrive(bar);
}
// The same from a thread that has read what it was to read (tcgen05.wait::ld) and has written
// nothing that the barrier is to publish.  A release would wait for its earlier global stores,
// about a microsecond.
template <bool kTma>
__device__ __forceinline__ void arrive_leader_read(uint32_t bar) {
  if constexpr (kTma)
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_leader(bar))
                 : "memory");
  else
    sm100::mbar_arrive(bar);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Boxes of a pair's block, complete at a barrier of either block.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const void* map, int c0, int c1,
                                             uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const void* map, int c0, int c1, int c2,
                                             uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}

// One look at phase `parity` of a barrier.  kOthers: what threads of the pair's other block have
// written before they arrived is to be seen (an acquire of the cluster's scope, which a wait for
// copies, MMAs or this block does without).
template <bool kOthers>
__device__ __forceinline__ bool product_try(uint32_t bar, uint32_t parity) {
  if (!kOthers) return sm100::mbar_try_wait(bar, parity);
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Looks until `look` finds what it waits for; false when *abort is set, or when *progress has
// stood still for `cycles` of `clock`.  What is waited for may take any number of stages (a part of
// a tile, or for a turn in the queue several), so that time alone says nothing.
#pragma nv_exec_check_disable
template <typename Look, typename Clock>
__host__ __device__ __forceinline__ bool wait_while_moving(Look look, Clock clock,
                                                           const volatile int* abort,
                                                           const volatile uint32_t* progress,
                                                           int64_t cycles) {
  if (look()) return true;
  int64_t t0 = clock();
  uint32_t seen = *progress;
  for (uint32_t i = 1;; ++i) {
    if (look()) return true;
    if ((i & 3u) != 0) continue;
    if (*abort) return false;
    const int64_t t = clock();
    if (t - t0 <= cycles) continue;
    const uint32_t now = *progress;
    if (now == seen) return false;
    seen = now, t0 = t;
  }
}
// Time is counted in the multiprocessor's cycles, which take far less to read than the clock.
template <bool kOthers = false>
__device__ __forceinline__ bool product_wait(uint32_t bar, uint32_t parity,
                                             const volatile int* abort,
                                             const volatile uint32_t* progress, int64_t cycles) {
  return wait_while_moving([&] { return product_try<kOthers>(bar, parity); },
                           [] { return (int64_t)clock64(); }, abort, progress, cycles);
}

// ---- the epilogue's chunks: 32 lanes (features) x 32 columns (rows) of a tile.

// Registers 8 j + i of column octet j: lanes lane / 4 + 8 (i / 2), columns 2 (lane % 4) + i % 2.
__device__ __forceinline__ void tmem_ld_fragments(uint32_t taddr, float (&v)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[4 * h]), "=r"(r[4 * h + 1]), "=r"(r[4 * h + 2]), "=r"(r[4 * h + 3]),
          "=r"(r[4 * h + 8]), "=r"(r[4 * h + 9]), "=r"(r[4 * h + 10]), "=r"(r[4 * h + 11]),
          "=r"(r[4 * h + 16]), "=r"(r[4 * h + 17]), "=r"(r[4 * h + 18]), "=r"(r[4 * h + 19]),
          "=r"(r[4 * h + 24]), "=r"(r[4 * h + 25]), "=r"(r[4 * h + 26]), "=r"(r[4 * h + 27])
        : "r"(taddr + ((uint32_t)(16 * h) << 16))
        : "memory");
  sm100::tmem_wait_ld();
}
// Adds the accumulator `from` to `to`, for the lanes and the chunks of columns (kChunk of them,
// kStep apart) that a warp stores; kAtATime columns in registers.
template <int kAtATime, int kChunk, int kStep>
__device__ __forceinline__ void add_part(uint32_t to, uint32_t from, int first, int n) {
  for (int c = first; c < n; c += kStep) {
#pragma unroll 1
    for (int i = 0; i < kChunk; i += kAtATime) {
      float a[kAtATime], b[kAtATime];
      uint32_t* x = reinterpret_cast<uint32_t*>(a);
      uint32_t* y = reinterpret_cast<uint32_t*>(b);
      if constexpr (kAtATime == 16) {
        sm100::tmem_ld16(to + c + i, x);
        sm100::tmem_ld16(from + c + i, y);
      } else {
        sm100::tmem_ld8(to + c + i, x);
        sm100::tmem_ld8(from + c + i, y);
      }
      sm100::tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < kAtATime; ++k) a[k] += b[k];
      if constexpr (kAtATime == 16)
        sm100::tmem_st16(to + c + i, x);
      else
        sm100::tmem_st8(to + c + i, x);
    }
  }
  sm100::tmem_wait_st();
}
__device__ __forceinline__ void clear(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.0f;
}

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  typename PairOf<T>::type p;
  pair_from_f32(p, a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// A storing warp's 2 KB, in which a chunk is turned over: a row's 32 features are four 16-byte
// blocks, exchanged so that neither the transposing stores nor the loads meet in a bank.
struct Turn {
  uint32_t base, put, get;
  __device__ __forceinline__ Turn(uint32_t at, int lane)
      : base(at),
        // lanes 8 b .. 8 b + 7 give the places of block b of rows 0 .. 7
        put(at + lane % 8 * 64 + ((lane / 8 ^ (lane >> 1 & 3)) << 4)),
        // lanes 4 r .. 4 r + 3 read row r
        get(at + lane / 4 * 64 + ((lane % 4 ^ (lane >> 3 & 3)) << 4)) {}
};

// Rounds kOctets octets of columns and stores them as `cols` rows of out, `stride` elements
// apart, from feature m on, as far as M.
template <typename T, int kOctets = 4>
__device__ __forceinline__ void store_chunk(const ProductArgs& A, const Turn& turn,
                                            const float (&v)[8 * kOctets], uint16_t* out,
                                            int64_t stride, int64_t row, int cols, int m, int M,
                                            int lane) {
  __syncwarp();
#pragma unroll
  for (int j = 0; j < kOctets; ++j)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                     turn.put + 512 * j),
                 "r"(pack_pair<T>(v[8 * j], v[8 * j + 1])),
                 "r"(pack_pair<T>(v[8 * j + 2], v[8 * j + 3])),
                 "r"(pack_pair<T>(v[8 * j + 4], v[8 * j + 5])),
                 "r"(pack_pair<T>(v[8 * j + 6], v[8 * j + 7]))
                 : "memory");
  __syncwarp();
  if (A.vec) {
    m += lane % 4 * 8;
    if (m < M) {
      uint16_t* to = out + (row + lane / 4) * stride + m;
      if (cols >= 8 * kOctets) {
#pragma unroll
        for (int i = 0; i < kOctets; ++i, to += 8 * stride)
          *reinterpret_cast<uint4*>(to) = sm100::lds128(turn.get + 512 * i);
      } else {
        for (int i = 0; 8 * i + lane / 4 < cols; ++i, to += 8 * stride)
          *reinterpret_cast<uint4*>(to) = sm100::lds128(turn.get + 512 * i);
      }
    }
  } else if (m + lane < M) {
    uint16_t* to = out + row * stride + m + lane;
    for (int r = 0; r < 8 * kOctets && r < cols; ++r, to += stride) {
      uint16_t w;
      asm volatile("ld.shared.u16 %0, [%1];"
                   : "=h"(w)
                   : "r"(turn.base + r * 64 + ((lane / 8 ^ (r >> 1 & 3)) << 4) + lane % 8 * 2)
                   : "memory");
      *to = w;
    }
  }
}

// A lane's kCount values, 64 bytes, as a half of its row of the warp's box.
template <typename T, int kCount>
__device__ __forceinline__ void put_row(uint32_t box, const float (&v)[32], int first, int half,
                                        int lane) {
  constexpr int kPer = 16 / (int)sizeof(T);
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    Packed<T, kPer> p;
    float f[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) f[k] = v[first + b * kPer + k];
    p.pack(f);
    sm100::sts128(box + lane * 128 + ((4 * half + b ^ (lane & 7)) << 4),
                  *reinterpret_cast<const uint4*>(&p));
  }
}

// Without the tensor memory accelerator: `rows` x `cols` of the chunk, turned by way of the box
// (fp32) so that a warp's lanes store neighbours.
template <typename T>
__device__ __forceinline__ void store_rows(T* to, int64_t stride, uint32_t box, const float (&v)[32],
                                           int rows, int cols, int lane) {
  __syncwarp();
  put_row<float, 16>(box, v, 0, 0, lane);
  put_row<float, 16>(box, v, 16, 1, lane);
  __syncwarp();
#pragma unroll 4
  for (int r = 0; r < rows && lane < cols; ++r, to += stride) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];"
                 : "=f"(f)
                 : "r"(box + r * 128 + ((lane / 4 ^ (r & 7)) << 4) + lane % 4 * 4)
                 : "memory");
    to[lane] = from_f32<T>(f);
  }
  __syncwarp();  // the next load from TMEM is the whole warp's
}

// By a whole warp: its box in shared memory as rows m .. m + 31 of an expert's result, from
// column n on, as far as the result goes; and the wait until the box may be written again.
__device__ __forceinline__ void box_store(const void* map, uint32_t box, int n, int m, int expert,
                                          int lane) {
  sm100::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(n), "r"(m), "r"(expert), "r"(box)
        : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
__device__ __forceinline__ void box_free(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}
__device__ __forceinline__ void box_end(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Zeros in elements first .. end - 1, by all threads; vec: both are multiples of 8, and the
// first element starts on 16 bytes.
__device__ __forceinline__ void clear_elements(void* out, int64_t first, int64_t end, bool vec,
                                               int64_t thread, int64_t threads) {
  if (vec)
    for (int64_t i = first / 8 + thread; i < end / 8; i += threads)
      static_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
  else
    for (int64_t i = first + thread; i < end; i += threads) static_cast<uint16_t*>(out)[i] = 0;
}

// Barrier `id` over `count` threads of whole warps, and whether all of them say yes.
__device__ __forceinline__ bool barrier_all(uint32_t id, uint32_t count, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((uint32_t)yes)
      : "memory");
  return r != 0;
}

constexpr int kProductThreads(int ctas, ProductMode mode) {
  return (4 + kStorers(ctas) +
          (ctas == 1 ? kProducers : mode == ProductMode::kWeight ? 1 : 0)) * 32;
}

// Warps: 0 copies, 1 MMAs, 2 tells the tiles, 3 and the last zero behind experts' last rows
// (dweight; they take turns, since one takes about 2 us from a stage's arrival to the next),
// 4 on store, and behind them kProducers load where loads are plain.
template <int kCtas, ProductMode kMode>
__global__ void __launch_bounds__(kProductThreads(kCtas, kMode), 1)
    hcmix_product_kernel(const __grid_constant__ ProductArgs A) {
  using namespace sm100;
  begin_kernel();
  constexpr bool kTma = kCtas > 1;
  constexpr bool kAcross = kMode != ProductMode::kRowsK;   // A lies with m contiguous
  constexpr bool kWeight = kMode == ProductMode::kWeight;  // and B with n
  constexpr int kDepth = kStages(kCtas);
  constexpr int kStore = kStorers(kCtas), kTurns = kStore * kTurnBytes(kMode);
  extern __shared__ uint8_t product_shared[];
  const uint32_t raw = smem_u32(product_shared);
  const uint32_t stages = (raw + 1023) & ~1023u;
  uint8_t* after = product_shared + (stages - raw) + kDepth * kStageBytes(kCtas);
  float* exchange = reinterpret_cast<float*>(after);
  ProductControl& C = *reinterpret_cast<ProductControl*>(after + kTurns + kRawBytes(kCtas));
  int* cum = reinterpret_cast<int*>(&C + 1);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int rank = blockIdx.x % kCtas;
  const bool leader = rank == 0;  // of a pair

  if (tid == 0) {
    const int takers = kStore + (kTma ? 1 : kProducers) + leader + (kTma && kWeight ? 2 : 0);
    for (int q = 0; q < kQueue; ++q) {
      mbar_init(smem_u32(&C.told[q]), 1);
      mbar_init(smem_u32(&C.taken[q]), takers);
    }
    for (int s = 0; s < kDepth; ++s) {
      mbar_init(smem_u32(&C.full[s]), kTma ? 1 : kProducers);
      mbar_init(smem_u32(&C.empty[s]), 1);
      mbar_init(smem_u32(&C.tail[s]), 1);
      mbar_init(smem_u32(&C.ready[s]), 2 * kCtas);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&C.acc_full[b]), 1);
      mbar_init(smem_u32(&C.acc_empty[b]), kStore * kCtas);
    }
    mbar_init(smem_u32(&C.drain), 1);
    C.abort = 0;
    C.copied = 0;
    fence_mbarrier_init();
  }
  // the pair's barriers are there before its other block touches them
  if (kTma) cluster_sync();
  if (warp == 2) product_tmem_alloc<kTma>(smem_u32(&C.tmem));
  if (!kWeight) count_tiles<kCtas>(A, cum, C.scan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem;
  const volatile int* abort = &C.abort;
  const volatile uint32_t* progress = &C.copied;
  const auto moved = [&](uint32_t n) { *const_cast<volatile uint32_t*>(progress) = n; };
  const auto gave_up = [&]() {
    record_device_error(&g_product_error, kDevWaitTimeout);
    *reinterpret_cast<volatile int*>(&C.abort) = 1;
    return false;
  };
  const auto wait = [&](uint64_t& bar, uint32_t parity) {
    return product_wait(smem_u32(&bar), parity, abort, progress, kProductWait) || gave_up();
  };
  const auto finish = [&](uint64_t& bar, uint32_t parity) {  // also after an abort
    const int none = 0;
    return product_wait(smem_u32(&bar), parity, &none, progress, kProductWait / 4);
  };
  // The next tile, by a whole warp; false behind the last, and after an abort.
  uint32_t turns = 0;
  const auto next = [&](ProductTile& T) {
    const int q = turns % kQueue;
    if (!__all_sync(0xffffffffu, wait(C.told[q], (turns / kQueue) & 1))) return false;
    T = C.tile[q];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&C.taken[q]));
    ++turns;
    return T.n > 0;
  };
  ProductTile T;

  if (!kTma && warp >= 4 + kStore) {
    // ---- plain loads: rows 16 p .. 16 p + 15 of a stage's 128 of A and 128 of B
    const int p = warp - (4 + kStore), half = p / 4 % 2;
    const bool of_a = p < kProducers / 2, flat = of_a ? kAcross : kWeight;  // flat: rows are k
    const uint32_t ring = smem_u32(after + kTurns) + p * (kRawDepth * kRawBox);
    RawRows* slots = C.raw[p];
    const Matrix3& X = of_a ? A.a : A.b;
    const int64_t apart = of_a && !kWeight ? X.expert : 0;
    const char* low = static_cast<const char*>(X.p);
    const char* high = low + 2 * ((A.E - 1) * apart + (int64_t)(X.outer - 1) * X.row + X.inner);
    uint32_t copied = 0, placed = 0;
    int kb = 0, blocks = 0;
    bool more = true;
    // A stage's blocks lie `step` bytes behind the one's before, a multiple of 16 either way
    // (128, or 64 rows of an even number of bytes), so that a tile's addresses are found once.
    // Rows that are not there are features or rows whose results are not stored, unless they
    // are k; elements behind a row's end are masked when they are placed.
    constexpr int kTurnsOfCopy = (kRawRows * 9 + 31) / 32;
    const char* from[kTurnsOfCopy];
    RawRows R;
    int64_t step = 0;
    bool idle = false;
    bool inside = false;  // all blocks of the tile's rows lie in the matrix
    // Copies one stage; false where there is none, or where its tile has not been told yet and
    // `may_wait` is not set: the tile is told when the MMA and storing warps have taken earlier
    // ones, for which they may need a stage that this warp has copied and not yet placed.
    const auto copy = [&](bool may_wait) {
      while (kb == blocks) {
        const bool told = mbar_test_wait(smem_u32(&C.told[turns % kQueue]), (turns / kQueue) & 1);
        if (!may_wait && !__all_sync(0xffffffffu, told)) return false;
        more = next(T);
        if (!more) return false;
        kb = 0;
        blocks = (T.depth + kTileK - 1) / kTileK;
        const int first = of_a ? (half ? T.m1 : T.m0) : T.n0 + 64 * half;  // feature or row
        const int inner = flat ? first : T.k0, outer = (flat ? T.k0 : first) + kRawRows * (p % 4);
        const int end = flat ? T.k0 + T.depth : of_a ? X.outer : T.n0 + T.n;
        R.at = low + 2 * (T.expert * apart + outer * X.row + inner);
        R.pitch = 2 * X.row;
        R.elements = X.inner - inner;
        R.rows = end - outer;
        // rows of B that nothing is computed from: a tile of few rows
        idle = !of_a && !flat && R.rows <= 0;
        step = flat ? kTileK * R.pitch : 2 * kTileK;
        const char* base = align16(R.at);
        const int rows = flat || R.rows > kRawRows ? kRawRows : R.rows;
        inside = base >= low &&
                 R.at + (blocks - 1 - flat) * step + (rows - 1) * R.pitch + kRawPitch <= high;
#pragma unroll
        for (int i = 0; i < kTurnsOfCopy; ++i) {
          const int at = i * 32 + lane, row = at / 9;
          from[i] = align16(R.at + row * R.pitch) + 16 * (at - 9 * row);
          if (row >= kRawRows || (!flat && row >= R.rows)) from[i] = nullptr;
        }
      }
      {
        const int slot = copied++ % kRawDepth;
        const uint32_t raw = ring + slot * kRawBox;
        if (idle) {
        } else if (inside && !(flat && kb == blocks - 1)) {
          const int64_t off = kb * step;
#pragma unroll
          for (int i = 0; i < kTurnsOfCopy; ++i)
            if (from[i] != nullptr)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                               raw + (i * 32 + lane) * 16),
                           "l"(from[i] + off)
                           : "memory");
        } else {
          RawRows now = R;
          now.at += kb * step;
          if (flat) now.rows -= kb * kTileK;
          else now.elements -= kb * kTileK;
          copy_raw(raw, now, low, high, lane);
        }
        if (lane == 0) {
          RawRows& told = slots[slot];
          told.at = R.at;
          told.pitch = R.pitch;
          told.elements = flat ? R.elements : R.elements - kb * kTileK;
          told.rows = !idle;
        }
        ++kb;
      }
      async_commit();
      return true;
    };
    for (;; ++placed) {
      while (more && copied - placed < kRawDepth && copy(copied == placed)) {
      }
      if (placed == copied) break;
      if (copied - placed == kRawDepth)
        async_wait<kRawDepth - 1>();
      else
        async_wait<0>();
      __syncwarp();
      const int s = placed % kDepth, slot = placed % kRawDepth;
      if (placed >= kDepth &&
          !__all_sync(0xffffffffu, wait(C.empty[s], (placed / kDepth - 1) & 1)))
        break;
      if (slots[slot].rows != 0) {
        place_raw(stages + s * kStageBytes(kCtas) + p * (kRawRows * 128), ring + slot * kRawBox,
                  slots[slot], lane);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&C.full[s]));
      if (p == 0 && lane == 0) moved(placed + 1);
    }
    async_wait<0>();
  } else if (kTma && warp == 0) {
    // ---- producer
    uint32_t it = 0;  // stages filled
    uint32_t full_at = 0, tail_at = 0, tails = 0;  // a bit for each stage: phases, and the last use
    bool ok = true;
    while (ok && next(T)) {
      const int blocks = (T.depth + kTileK - 1) / kTileK;
      const int n = round_rows<kCtas>(T.n) / kCtas;  // this block's share of B
      const int n0 = T.n0 + rank * n;
      const int place = kTma && kWeight ? tail_place(T.depth) : blocks;
      for (int i = 0; ok && i < blocks; ++i, ++it) {
        const int s = it % kDepth;
        const int kb = i < place ? i : i == place ? blocks - 1 : i - 1;
        const uint32_t a = stages + s * kStageBytes(kCtas), b = a + kABytes;
        const int k = T.k0 + kb * kTileK;
        if (it >= kDepth) ok = wait(C.empty[s], (it / kDepth - 1) & 1);
        if (!ok) break;
        if constexpr (kTma) {
          if (lane == 0) {
            moved(it + 1);
            const int boxes = (n + 63) / 64;
            const uint32_t bytes = kABytes + (kWeight ? boxes * kBoxBytes : n * 128);
            // (without the hint these copies, and what runs behind them, take the same time
            // within 2 %: 128 experts of 256 rows 488 us either way, a call behind 2.7 GB 96 us)
            const uint64_t keep = l2_policy_evict_last();
            // block 0 waits for both blocks' copies at once, but for the last rows of an expert,
            // behind which each block has to zero its own
            const bool tail = i == place;
            const uint32_t own = smem_u32(tail ? &C.tail[s] : &C.full[s]);
            const uint32_t bar = tail ? own : in_leader(own);
            if (tail)
              mbar_arrive_expect_tx(own, bytes);
            else if (leader)
              mbar_arrive_expect_tx(own, 2 * bytes);
            (tail ? tail_at : full_at) ^= 1u << s;
            tails = (tails & ~(1u << s)) | (uint32_t)tail << s;
            for (int h = 0; h < 2; ++h) {
              const int m = h ? T.m1 : T.m0;
              if (kWeight)
                pair_load_2d(a + h * kBoxBytes, &A.a_map, m, k, bar, keep);
              else if (kAcross)
                pair_load_3d(a + h * kBoxBytes, &A.a_map, m, k, T.expert, bar, keep);
              else
                pair_load_3d(a + h * kBoxBytes, &A.a_map, k, m, T.expert, bar, keep);
            }
            if (kWeight) {
              for (int j = 0; j < boxes; ++j)
                pair_load_2d(b + j * kBoxBytes, &A.b_map, n0 + j * 64, k, bar, keep);
            } else {
              int r = 0;
              for (; r + 64 <= n; r += 64)
                pair_load_2d(b + r * 128, &A.b_map, k, n0 + r, bar, keep);
              for (; r < n; r += 16)
                pair_load_2d(b + r * 128, &A.b16_map, k, n0 + r, bar, keep);
            }
          }
          __syncwarp();
        }
      }
    }
    if (kTma && lane == 0) {
      // copies that nobody waited for (another role gave up) land before the block ends
      for (uint32_t last = it > kDepth ? it - kDepth : 0; last < it; ++last) {
        const int s = last % kDepth;
        if (tails >> s & 1)
          finish(C.tail[s], ~(tail_at >> s) & 1);
        else if (leader)
          finish(C.full[s], ~(full_at >> s) & 1);
      }
      // and so do the MMAs' arrivals here, which are on their own when the leader's warp is done:
      // each one's, since none orders the others (after an abort as far as there are any)
      bool come = true;
      for (uint32_t last = it > kDepth ? it - kDepth : 0; come && last < it; ++last)
        come = finish(C.empty[last % kDepth], (last / kDepth) & 1);
      finish(C.drain, 0);
    }
  } else if (kTma && kWeight && (warp == 3 || warp == 4 + kStore)) {
    // ---- the last stage of an expert took rows of the next one along: they count as zeros
    uint32_t it = 0, tail_at = 0, tails = 0;
    bool ok = true;
    while (ok && next(T)) {
      const int left = T.depth % kTileK, s = (it + tail_place(T.depth)) % kDepth;
      it += (T.depth + kTileK - 1) / kTileK;
      if (left == 0) continue;
      // Both warps wait for every stage, and the MMAs for both warps: a wait by parity takes a
      // phase for another if its barrier is not the phase before, or is two ahead.
      ok = __all_sync(0xffffffffu, wait(C.tail[s], tail_at >> s & 1));
      tail_at ^= 1u << s;
      if (!ok) break;
      if ((tails++ & 1) != (warp == 3 ? 0u : 1u)) {  // the other's turn
        if (lane == 0) arrive_leader_read<kTma>(smem_u32(&C.ready[s]));
        continue;
      }
      const int boxes = 2 + (round_rows<kCtas>(T.n) / kCtas + 63) / 64;
      // of the last 16 rows that the MMA reads
      const uint32_t from = left * 128 + lane * 16, to = (left + 15) / 16 * 16 * 128;
      for (int i = 0; i < boxes; ++i)
        for (uint32_t at = from; at < to; at += 512)
          sts128(stages + s * kStageBytes(kCtas) + i * kBoxBytes + at, make_uint4(0, 0, 0, 0));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_leader<kTma>(smem_u32(&C.ready[s]));
    }
  } else if (warp == 1 && leader) {
    // ---- MMA
    uint32_t it = 0, full_at = 0, tail_at = 0;
    uint32_t first = 1, acc_at = 0, acc_used = 0;  // accumulators: see the epilogue
    uint32_t empty_at = 0, used = 0;  // a bit for each stage: its arrivals so far, and whether any
    constexpr uint32_t kPair = (1u << kCtas) - 1;
    bool ok = true;
    const uint32_t kind = A.f16 ? 0u : (1u << 7) | (1u << 10);
    while (ok && next(T)) {
      const int blocks = (T.depth + kTileK - 1) / kTileK;
      if (blocks == 0) continue;
      const uint32_t idesc = (1u << 4) | kind | (kAcross ? 1u << 15 : 0u) |
                             (kWeight ? 1u << 16 : 0u) |
                             ((uint32_t)(round_rows<kCtas>(T.n) >> 3) << 17) |
                             ((uint32_t)(kTileM * kCtas >> 4) << 24);
      if (T.part & kFirstPart) first ^= 1;
      const uint32_t buf = T.part & kFirstPart ? first : first ^ 1;
      if (acc_used >> buf & 1)
        ok = __all_sync(0xffffffffu, wait(C.acc_empty[buf], ~(acc_at >> buf) & 1));
      acc_at ^= 1u << buf, acc_used |= 1u << buf;
      tc_fence_after();
      const uint32_t d = tmem + buf * kAccumulator;
      const int place = kTma && kWeight ? tail_place(T.depth) : blocks;
      for (int kb = 0; ok && kb < blocks; ++kb) {
        const bool tail = place < blocks && kb == blocks - 1;
        const int s = (it + (tail ? place : kb < place ? kb : kb + 1)) % kDepth;
        const int left = T.depth - kb * kTileK;
        ok = tail ? product_wait<true>(smem_u32(&C.ready[s]), tail_at >> s & 1, abort, progress,
                                       kProductWait) ||
                        gave_up()
                  : wait(C.full[s], full_at >> s & 1);
        ok = __all_sync(0xffffffffu, ok);
        (tail ? tail_at : full_at) ^= 1u << s;
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = stages + s * kStageBytes(kCtas), b = a + kABytes;
        const uint64_t da = kAcross ? desc_mn_sw128(a) : smem_desc_sw128(a);
        const uint64_t db = kWeight ? desc_mn_sw128(b) : smem_desc_sw128(b);
        // 16 k: 32 bytes of a row, or 16 rows
        constexpr int kA = kAcross ? 128 : 2, kB = kWeight ? 128 : 2;
        if (left >= kTileK) {
          mma_64<kTma, kA, kB>(d, da, db, idesc, kb > 0);
        } else {
          for (int i = 0; i * 16 < left; ++i)
            mma_16<kTma>(d, da + i * kA, db + i * kB, idesc, kb > 0 || i > 0);
        }
        mma_commit<kTma>(smem_u32(&C.empty[s]), kPair);
        empty_at ^= 1u << s, used |= 1u << s;
        if (kb == blocks - 1) mma_commit<kTma>(smem_u32(&C.acc_full[buf]), kPair);
      }
      it += blocks;
    }
    // what was issued is done, and has arrived here, before the block ends
    mma_commit<kTma>(smem_u32(&C.drain), kPair);
    for (int s = 0; s < kDepth; ++s)
      if (used >> s & 1) finish(C.empty[s], ~(empty_at >> s) & 1);
    finish(C.drain, 0);
  } else if (warp >= 4 && warp < 4 + kStore) {
    // ---- epilogue: TMEM lanes 32 * w on, chunks of 32 columns in turn.  A tile's first part is in
    // the accumulator that the tile before did not begin with, and is stored from there with the
    // others, which come one after the other in the other one, added.
    const int w = warp % 4, half = (warp - 4) / 4;
    const int bar = 1 + (w & 1) + 2 * half;  // of g's and u's warp
    uint32_t first = 1, acc_at = 0;
    bool ok = true;
    float* mine = exchange + (warp - 4) * (kTurnBytes(kMode) / 4);
    const float* other = exchange + (half * 4 + (w ^ 2)) * (kTurnBytes(kMode) / 4);
    const Turn turn(smem_u32(mine), lane);
    const auto store_tiles = [&](auto zero) {
      using T16 = decltype(zero);
      for (;;) {
        // g's and u's warps go on together, or both leave
        bool have = next(T);
        if (A.gated) have = barrier_all(bar, 64, have);
        if (!have) break;
        const bool any = T.depth > 0;
        uint32_t buf = 0;
        if (any) {
          if (T.part & kFirstPart) first ^= 1;
          buf = T.part & kFirstPart ? first : first ^ 1;
          ok = wait(C.acc_full[buf], acc_at >> buf & 1);
          acc_at ^= 1u << buf;
          ok = A.gated ? barrier_all(bar, 64, ok) : __all_sync(0xffffffffu, ok);
        }
        if (!ok) break;
        tc_fence_after();
        const auto give_back = [&](uint32_t which) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_leader_read<kTma>(smem_u32(&C.acc_empty[which]));
        };
        const uint32_t lanes = tmem + ((uint32_t)(w * 32) << 16);
        const uint32_t d = lanes + first * kAccumulator;
        if (!(T.part & kFirstPart)) {
          constexpr int kChunk = kWeight ? 64 : 32;
          add_part<kTma ? 16 : 8, kChunk, kChunk * kStore / 4>(d, lanes + buf * kAccumulator,
                                                                kChunk * half, T.n);
          give_back(buf);
        }
        if (!(T.part & kLastPart)) continue;
        if constexpr (kWeight) {
          const int m0 = T.m0 + w * 32;
          for (int c = 64 * half; c < T.n && m0 < A.M; c += 16 * kStore) {
            if (A.vec) box_free(lane);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v[32];
              if (any) {
                tmem_ld32(d + c + 32 * h, reinterpret_cast<uint32_t(&)[32]>(v));
                tmem_wait_ld();
              } else {
                clear(v);
              }
              const int n = T.n0 + c + 32 * h, cols = A.N - n < 32 ? A.N - n : 32;
              if (!A.vec) {
                const int64_t at = ((int64_t)T.expert * A.M + m0) * A.N + n;
                const int rows = A.M - m0 < 32 ? A.M - m0 : 32;
                if (A.out_f32)
                  store_rows(static_cast<float*>(A.out) + at, A.N, turn.base, v, rows, cols, lane);
                else
                  store_rows(static_cast<T16*>(A.out) + at, A.N, turn.base, v, rows, cols, lane);
              } else if (A.out_f32) {  // a box of 32 columns
                put_row<float, 16>(turn.base, v, 0, 0, lane);
                put_row<float, 16>(turn.base, v, 16, 1, lane);
                if (cols > 0) box_store(&A.out_map, turn.base, n, m0, T.expert, lane);
                if (h == 0) box_free(lane);
              } else {
                put_row<T16, 32>(turn.base, v, 0, h, lane);
                if (h == 1) box_store(&A.out_map, turn.base, n - 32, m0, T.expert, lane);
              }
            }
          }
        } else {
          const int64_t row = T.n0;
          for (int c = 32 * half; c < T.n; c += 8 * kStore) {
            const int cols = T.n - c < 32 ? T.n - c : 32;
            float v[32];
            if (any)
              tmem_ld_fragments(d + c, v);
            else
              clear(v);
            if (!A.gated) {
              store_chunk<T16>(A, turn, v, static_cast<uint16_t*>(A.out), A.M, row + c, cols,
                          T.m0 + w * 32, A.M, lane);
            } else {
              const int f = T.m0 + (w & 1) * 32;
              if (A.saved != nullptr)
                store_chunk<T16>(A, turn, v, static_cast<uint16_t*>(A.saved) + (w < 2 ? 0 : A.M),
                            2 * (int64_t)A.M, row + c, cols, f, A.M, lane);
              // g's warps give their upper 16 columns to u's, and get the lower ones of u
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 16; ++i) mine[i * 32 + lane] = w < 2 ? v[16 + i] : v[i];
              named_bar_sync(bar, 64);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float o = other[i * 32 + lane];
                v[i] = w < 2 ? gate(v[i], o) : gate(o, v[16 + i]);
              }
              named_bar_sync(bar, 64);  // both have read
              const int c0 = w < 2 ? 0 : 16;
              store_chunk<T16, 2>(A, turn, reinterpret_cast<float(&)[16]>(v),
                             static_cast<uint16_t*>(A.out), A.M, row + c + c0, cols - c0, f, A.M, lane);
            }
          }
        }
        if (any) give_back(first);
      }
    };
    if (A.f16)
      store_tiles(__half{});
    else
      store_tiles(__nv_bfloat16{});
    if (kWeight && A.vec) box_end(lane);
  } else if (warp == 2) {
    // ---- the tiles, in turn over the clusters.  Finding one takes loads and divisions, about
    // a microsecond: the lanes find 32 at a time.
    const int64_t tiles = tile_count<kCtas, kMode>(A, cum), step = gridDim.x / kCtas;
    bool ok = true, more = true;
    for (int64_t t0 = blockIdx.x / kCtas; ok && more; t0 += 32 * step) {
      const int64_t t = t0 + lane * step;
      if (t < tiles) T = tile_at<kCtas, kMode>(A, cum, t, rank);
      else T = {};
      const int parts = T.depth > 0 ? (T.depth - 1) / A.part + 1 : 1;
      for (int i = 0; ok && more && i < 32; ++i) {
        const int of = __shfl_sync(0xffffffffu, parts, i);
        for (int p = 0; ok && p < of; ++p, ++turns) {
          const int q = turns % kQueue;
          if (turns >= kQueue)
            ok = __all_sync(0xffffffffu, wait(C.taken[q], (turns / kQueue - 1) & 1));
          if (!ok) break;
          if (lane == i) {
            C.tile[q] = T;
            C.tile[q].part = (p == 0 ? kFirstPart : 0) | (p == of - 1 ? kLastPart : 0);
            if (T.depth > A.part) {
              C.tile[q].depth = A.part;
              T.k0 += A.part, T.depth -= A.part;  // of the next part
            }
            mbar_arrive(smem_u32(&C.told[q]));
          }
        }
        more = __shfl_sync(0xffffffffu, T.n, i) > 0;
      }
    }
  }
  // rows that no expert has
  if (!kWeight) {
    const int64_t end = clamp_offset(A.offsets[A.E], A.R);
    const int64_t from = (int64_t)blockIdx.x * blockDim.x + tid;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    clear_elements(A.out, end * A.M, A.R * A.M, A.vec, from, step);
    if (A.saved != nullptr) clear_elements(A.saved, end * 2 * A.M, A.R * 2 * A.M, A.vec, from, step);
  }
  tc_fence_before();
  __syncthreads();
  // no block ends while the other's threads may still arrive at its barriers
  if (kTma) cluster_sync();
  tc_fence_after();
  if (warp == 2) product_tmem_dealloc<kTma>(tmem);
}

// ---- host side

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
  static EncodeFn fn = []() -> EncodeFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (checked(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                 cudaEnableDefault, &q)) != HCMIX_OK ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Whether TMA can read the matrix: 16-byte rows, strides below 2^40 bytes.
inline bool tma_readable(const Matrix3& X, int experts) {
  const int64_t most = (int64_t)1 << 39;
  return reinterpret_cast<uintptr_t>(X.p) % 16 == 0 && X.row % 8 == 0 && X.row < most &&
         (experts <= 1 || (X.expert % 8 == 0 && X.expert < most));
}

// Boxes of 64 elements of `rows` rows, 128-byte swizzle, zeros outside.
inline bool make_box_map(CUtensorMap* map, const Matrix3& X, int experts, bool f16, uint32_t rows) {
  EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)X.inner, (cuuint64_t)X.outer, (cuuint64_t)experts};
  // the stride of a single expert is not used
  const cuuint64_t strides[2] = {(cuuint64_t)X.row * 2,
                                 (cuuint64_t)(experts == 1 ? X.row : X.expert) * 2};
  const cuuint32_t box[3] = {64, rows, 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
            experts == 0 ? 2 : 3, const_cast<void*>(X.p), dims, strides, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// dweight's boxes; false where its rows do not start on 16 bytes.
inline bool make_out_map(ProductArgs& A) {
  EncodeFn fn = encode_fn();
  const int size = A.out_f32 ? 4 : 2;
  const cuuint64_t row = (cuuint64_t)A.N * size, expert = row * A.M;
  if (fn == nullptr || row % 16 != 0 || reinterpret_cast<uintptr_t>(A.out) % 16 != 0) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)A.N, (cuuint64_t)A.M, (cuuint64_t)A.E};
  const cuuint64_t strides[2] = {row, expert};
  const cuuint32_t box[3] = {128u / size, 32, 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  const CUtensorMapDataType type = A.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : A.f16   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return fn(&A.out_map, type, 3, A.out, dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The clusters that the current device runs at a time.  Asked for once a device.
template <int kCtas, ProductMode kMode>
hcmix_status resident_clusters(int* clusters) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0, n = 0;
  hcmix_status st = checked(cudaGetDevice(&dev));
  if (st != HCMIX_OK) return st;
  const bool keep = dev >= 0 && dev < kDevices;
  if (keep && (n = known[dev].load(std::memory_order_relaxed)) > 0) {
    *clusters = n;
    return HCMIX_OK;
  }
  auto kernel = hcmix_product_kernel<kCtas, kMode>;
  const size_t smem = product_smem<kCtas, kMode>(kProductExperts);
  st = checked(
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  if (st != HCMIX_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(kProductThreads(kCtas, kMode));
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  st = checked(cudaOccupancyMaxActiveClusters(&n, kernel, &cfg));
  if (st != HCMIX_OK) return st;
  if (n < 1) return HCMIX_ERR_CUDA;
  if (keep) known[dev].store(n, std::memory_order_relaxed);
  *clusters = n;
  return HCMIX_OK;
}

template <int kCtas, ProductMode kMode>
hcmix_status launch_product(const ProductArgs& A, cudaStream_t stream) {
  int clusters = 0;
  const hcmix_status st = resident_clusters<kCtas, kMode>(&clusters);
  if (st != HCMIX_OK) return st;
  const int width = tile_width<kCtas>(A);
  const int64_t mt = (A.M + width - 1) / width;
  const int64_t tiles = kMode == ProductMode::kWeight
                            ? A.E * mt * ((A.N + kTileN(kCtas) - 1) / kTileN(kCtas))
                            : mt * (A.R / kTileN(kCtas) + (A.R < A.E ? A.R : A.E));
  const int64_t grid = tiles < clusters ? (tiles > 0 ? tiles : 1) : clusters;
  return launch(hcmix_product_kernel<kCtas, kMode>, dim3((unsigned)grid * kCtas),
                dim3(kProductThreads(kCtas, kMode)), product_smem<kCtas, kMode>(A.E),
                product_smem<kCtas, kMode>(kProductExperts), stream, A, kCtas);
}

// a, b, offsets, R, E, M, N, K, gated, out and types are set.
template <ProductMode kMode>
hcmix_status run_product(ProductArgs& A, cudaStream_t stream) {
  A.part = A.out_f32 ? kPartK32 : kPartK;
  if (kMode == ProductMode::kWeight) {
    A.vec = make_out_map(A);
  } else {
    A.vec = vector_bytes(2, {{A.out, A.M}, {A.saved, A.M}}) == 16;
    A.panel = panel_tiles(A.K);
  }
  const int experts = kMode == ProductMode::kWeight ? 0 : A.E;  // 0: a is a matrix as b is
  // a box starts on 16 bytes: u's features, too, where they lie along the rows
  const bool starts = kMode != ProductMode::kRowsM || !A.gated || A.M % 8 == 0;
  if (A.R > 0 && starts && tma_readable(A.a, experts) && tma_readable(A.b, 0) &&
      make_box_map(&A.a_map, A.a, experts, A.f16, 64) &&
      make_box_map(&A.b_map, A.b, 0, A.f16, 64) && make_box_map(&A.b16_map, A.b, 0, A.f16, 16))
    return launch_product<2, kMode>(A, stream);
  return launch_product<1, kMode>(A, stream);
}

}  // namespace sublayer
}  // namespace hcmix
