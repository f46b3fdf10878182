// Matrix products grouped by expert: the rows of each expert with its weights on
// the tensor cores, and the weights' gradients.
//
// One kernel computes transposed tiles D[m, n] = sum_k A[m, k] B[n, k], m an output
// feature (a TMEM lane) and n a row of the expert:
//
//   product            m: features of W[e]      n: rows of xs     k: width of xs
//   its dxs            m: width of W[e]         n: rows of dys    k: features
//   its dweight        m: inner index of dW[e]  n: its outer one  k: rows of the expert
//
// With the rows as the MMA's N, which may be any multiple of 16, an expert of few rows
// costs few columns and not a whole tile of 128; and a warp's lanes are neighbours in
// the row-major result.  fp32 accumulation in TMEM over all of k, one rounding at the
// store.  Blocks are persistent: a producer fills a ring of 64-wide slices of A and B,
// one thread issues the MMAs, and four warps store a tile while the next is computed.
#pragma once

#include <cuda.h>

#include "hcmix_common.cuh"
#include "hcmix_sm100.cuh"
#include "hcmix_vec.cuh"

namespace hcmix {
namespace sublayer {

constexpr int kProductExperts = 4096;
constexpr int kTileM = 128, kTileN = 256, kTileK = 64;
constexpr int kBoxBytes = 64 * 128;  // 64 rows of 64 16-bit elements
constexpr int kABytes = kTileM * kTileK * 2, kBBytes = kTileN * kTileK * 2;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kStages = 4;
constexpr int kPanel = 16;  // row tiles that take their turns at the same weights
constexpr uint64_t kProductWaitNs = 2000000000ull;

// One operand as it lies in memory: rows of contiguous elements.
struct Matrix3 {
  const void* p;
  int64_t row, expert;  // strides in elements
  int inner, outer;     // extents; rows of experts: outer is set by each tile
};

struct ProductArgs {
  CUtensorMap a_map, b_map, b16_map;  // boxes of 64 x 64, and of 64 x 16
  Matrix3 a, b;
  const int32_t* offsets;
  int64_t R;
  int E;
  int M, N, K;        // extents of m, n and k; product: N unused, dweight: K unused
  int gated;          // A's rows M .. 2 M - 1 are u's features, those before g's
  void* out;          // product: [R, M]; dweight: [E, N, M]
  void* saved;        // gated: [R, 2 M] or null
  int f16, out_f32;
};

enum class ProductMode { kRowsK, kRowsM, kWeight };  // A's contiguous index: k, m; dweight

static __device__ uint32_t g_product_error;

struct ProductControl {
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  int scan[32];
};
constexpr size_t kExchangeBytes = 4 * 16 * 32 * 4;  // gated: a half chunk of each warp
constexpr size_t product_smem(int E) {
  return 1024 + (size_t)kStages * kStageBytes + kExchangeBytes + sizeof(ProductControl) +
         ((size_t)E + 1) * 4 + 64;
}
static_assert(product_smem(kProductExperts) <= 227 * 1024, "shared memory of a block");

struct ProductTile {
  int expert;
  int m0, m1;     // origins of the two halves (64 lanes each) of A
  int64_t n0;     // first row of B, or first outer feature
  int n;          // valid ones
  int64_t k0;     // dweight: the expert's first row
  int64_t depth;  // of k
};

__device__ __forceinline__ int clamp_offset(int v, int64_t R) {
  return v < 0 ? 0 : v > R ? (int)R : v;
}
// The expert's rows, within 0 .. R whatever offsets holds.
__device__ __forceinline__ void expert_rows(const ProductArgs& A, int e, int& first, int& count) {
  first = clamp_offset(A.offsets[e], A.R);
  const int last = clamp_offset(A.offsets[e + 1], A.R);
  count = last > first ? last - first : 0;
}

// The number of row tiles of all experts before each, in `cum`.
__device__ __forceinline__ void count_tiles(const ProductArgs& A, int* cum, int* scan) {
  const int threads = blockDim.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int per = (A.E + threads - 1) / threads;
  const int e0 = tid * per < A.E ? tid * per : A.E, e1 = e0 + per < A.E ? e0 + per : A.E;
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    int first, count;
    expert_rows(A, e, first, count);
    const int tiles = (count + kTileN - 1) / kTileN;
    cum[e + 1] = tiles;
    sum += tiles;
  }
  int before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += t;
  }
  if (lane == 31) scan[warp] = before;
  __syncthreads();
  before -= sum;
  for (int w = 0; w < warp; ++w) before += scan[w];
  if (tid == 0) cum[0] = 0;
  for (int e = e0; e < e1; ++e) {
    before += cum[e + 1];
    cum[e + 1] = before;
  }
  __syncthreads();
}

template <ProductMode kMode>
__device__ __forceinline__ int64_t tile_count(const ProductArgs& A, const int* cum) {
  const int width = A.gated ? kTileM / 2 : kTileM;
  const int64_t mt = (A.M + width - 1) / width;
  if (kMode == ProductMode::kWeight) return A.E * mt * ((A.N + kTileN - 1) / kTileN);
  return cum[A.E] * mt;
}

template <ProductMode kMode>
__device__ __forceinline__ ProductTile tile_at(const ProductArgs& A, const int* cum, int64_t t) {
  ProductTile T;
  const int width = A.gated ? kTileM / 2 : kTileM;
  const int64_t mt = (A.M + width - 1) / width;
  int64_t m;
  if (kMode == ProductMode::kWeight) {
    const int64_t nt = (A.N + kTileN - 1) / kTileN;
    T.expert = (int)(t / (mt * nt));
    const int64_t rest = t - T.expert * (mt * nt);
    m = rest / nt;
    T.n0 = (rest - m * nt) * kTileN;
    T.n = A.N - T.n0 < kTileN ? (int)(A.N - T.n0) : kTileN;
    int first, count;
    expert_rows(A, T.expert, first, count);
    T.k0 = first, T.depth = count;
  } else {
    int lo = 0, hi = A.E;  // cum[lo] * mt <= t < cum[hi] * mt
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (cum[mid] * mt <= t) lo = mid; else hi = mid;
    }
    T.expert = lo;
    const int64_t local = t - cum[lo] * mt;
    const int nt = cum[lo + 1] - cum[lo];
    const int panel = (int)(local / (kPanel * mt));
    const int pn = nt - panel * kPanel < kPanel ? nt - panel * kPanel : kPanel;
    const int64_t rest = local - panel * (kPanel * mt);
    m = rest / pn;
    const int j = panel * kPanel + (int)(rest - m * pn);
    int first, count;
    expert_rows(A, lo, first, count);
    // the expert's tiles are of like size, so that none of them is nearly empty
    const int size = ((count + nt - 1) / nt + 15) / 16 * 16;
    T.n0 = first + (int64_t)j * size;
    T.n = count - j * size < size ? count - j * size : size;
    T.k0 = 0, T.depth = A.K;
  }
  T.m0 = (int)m * width;
  T.m1 = A.gated ? A.M + T.m0 : T.m0 + kTileM / 2;
  return T;
}

__device__ __forceinline__ int round16(int n) { return (n + 15) & ~15; }

// ---- plain loads: 64 x `rows` elements into the swizzled box at `dst`, element by
// element, zeros outside of the matrix.  For matrices whose rows do not all start on
// 16 bytes.
__device__ __forceinline__ void load_box(uint32_t dst, const Matrix3& X, int expert, int64_t inner0,
                                         int64_t outer0, int64_t outer_end, int rows, int tid,
                                         int threads) {
  const uint16_t* base = static_cast<const uint16_t*>(X.p) + expert * X.expert;
  for (int i = tid; i < rows * 8; i += threads) {
    const int r = i >> 3, c = i & 7;
    const int64_t outer = outer0 + r, inner = inner0 + c * 8;
    uint16_t v[8];
    const bool row_in = outer < outer_end;
    const uint16_t* p = base + outer * X.row + inner;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = row_in && inner + k < X.inner ? p[k] : (uint16_t)0;
    uint4 w;
    w.x = v[0] | (uint32_t)v[1] << 16, w.y = v[2] | (uint32_t)v[3] << 16;
    w.z = v[4] | (uint32_t)v[5] << 16, w.w = v[6] | (uint32_t)v[7] << 16;
    sm100::sts128(dst + r * 128 + ((c ^ (r & 7)) << 4), w);
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

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void store_value(void* out, int64_t at, float v, bool f32, bool f16) {
  if (f32)
    static_cast<float*>(out)[at] = v;
  else if (f16)
    static_cast<__half*>(out)[at] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
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

__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

constexpr int kProducers = 8;  // warps, where loads are plain
template <bool kTma>
constexpr int kProductThreads = kTma ? 256 : 256 + kProducers * 32;

template <bool kTma, ProductMode kMode>
__global__ void __launch_bounds__(kProductThreads<kTma>, 1)
    hcmix_product_kernel(const __grid_constant__ ProductArgs A) {
  using namespace sm100;
  begin_kernel();
  extern __shared__ uint8_t product_shared[];
  const uint32_t raw = smem_u32(product_shared);
  const uint32_t stages = (raw + 1023) & ~1023u;
  uint8_t* after = product_shared + (stages - raw) + kStages * kStageBytes;
  float* exchange = reinterpret_cast<float*>(after);
  ProductControl& C = *reinterpret_cast<ProductControl*>(after + kExchangeBytes);
  int* cum = reinterpret_cast<int*>(after + kExchangeBytes + sizeof(ProductControl));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  constexpr bool kAcross = kMode != ProductMode::kRowsK;    // A lies with m contiguous
  constexpr bool kWeight = kMode == ProductMode::kWeight;  // and B with n

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&C.full[s]), kTma ? 1 : kProducers);
      mbar_init(smem_u32(&C.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&C.acc_full[b]), 1);
      mbar_init(smem_u32(&C.acc_empty[b]), 4);
    }
    mbar_init(smem_u32(&C.drain), 1);
    C.abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&C.tmem), 512);
    tmem_relinquish();
  }
  if (!kWeight) count_tiles(A, cum, C.scan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem;
  const int64_t tiles = tile_count<kMode>(A, cum);
  const volatile int* abort = &C.abort;
  const auto wait = [&](uint64_t& bar, uint32_t parity) {
    if (mbar_wait(smem_u32(&bar), parity, abort, kProductWaitNs)) return true;
    record_device_error(&g_product_error, kDevWaitTimeout);
    *reinterpret_cast<volatile int*>(&C.abort) = 1;
    return false;
  };

  if (kTma ? warp == 0 : warp >= 8) {
    // ---- producer
    uint32_t it = 0;  // stages filled
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const ProductTile T = tile_at<kMode>(A, cum, t);
      const int blocks = (int)((T.depth + kTileK - 1) / kTileK);
      const int n16 = round16(T.n);
      for (int kb = 0; ok && kb < blocks; ++kb, ++it) {
        const int s = it % kStages;
        const uint32_t a = stages + s * kStageBytes, b = a + kABytes;
        const int64_t k = T.k0 + (int64_t)kb * kTileK;
        if (it >= kStages) ok = wait(C.empty[s], (it / kStages - 1) & 1);
        if (!ok) break;
        if constexpr (kTma) {
          if (lane == 0) {
            const uint32_t bar = smem_u32(&C.full[s]);
            const uint64_t keep = l2_policy_evict_last();
            const int nb = kWeight ? (n16 + 63) / 64 : 0;
            const uint32_t bytes = kABytes + (kWeight ? nb * kBoxBytes : n16 * 128);
            mbar_arrive_expect_tx(bar, bytes);
            for (int h = 0; h < 2; ++h) {
              const int m = h ? T.m1 : T.m0;
              if (kWeight)
                tma_load_2d(a + h * kBoxBytes, &A.a_map, m, (int)k, bar, keep);
              else if (kAcross)
                tma_load_3d(a + h * kBoxBytes, &A.a_map, m, (int)k, T.expert, bar, keep);
              else
                tma_load_3d(a + h * kBoxBytes, &A.a_map, (int)k, m, T.expert, bar, keep);
            }
            if (kWeight) {
              for (int i = 0; i < nb; ++i)
                tma_load_2d(b + i * kBoxBytes, &A.b_map, (int)T.n0 + i * 64, (int)k, bar, keep);
            } else {
              int r = 0;
              for (; r + 64 <= n16; r += 64)
                tma_load_2d(b + r * 128, &A.b_map, (int)k, (int)T.n0 + r, bar, keep);
              for (; r < n16; r += 16)
                tma_load_2d(b + r * 128, &A.b16_map, (int)k, (int)T.n0 + r, bar, keep);
            }
          }
          __syncwarp();
        } else {
          const int ptid = tid - 256;
          constexpr int pthreads = kProducers * 32;
          const int64_t k_end = T.k0 + T.depth;
          for (int h = 0; h < 2; ++h) {
            const int m = h ? T.m1 : T.m0;
            if (kAcross)
              load_box(a + h * kBoxBytes, A.a, T.expert, m, k, k_end, 64, ptid, pthreads);
            else
              load_box(a + h * kBoxBytes, A.a, T.expert, k, m, A.a.outer, 64, ptid, pthreads);
          }
          if (kWeight) {
            for (int i = 0; i * 64 < n16; ++i)
              load_box(b + i * kBoxBytes, A.b, 0, T.n0 + i * 64, k, k_end, 64, ptid, pthreads);
          } else {
            load_box(b, A.b, 0, k, T.n0, T.n0 + T.n, n16, ptid, pthreads);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&C.full[s]));
        }
      }
    }
    if (kTma) {
      // copies that nobody waited for (another role gave up) land before the block ends
      for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i) {
        const int none = 0;
        mbar_wait(smem_u32(&C.full[i % kStages]), (i / kStages) & 1, &none, kProductWaitNs / 4);
      }
    }
  } else if (warp == 1) {
    // ---- MMA
    uint32_t it = 0, acc = 0;
    bool ok = true;
    const uint32_t kind = A.f16 ? 0u : (1u << 7) | (1u << 10);
    for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const ProductTile T = tile_at<kMode>(A, cum, t);
      const int blocks = (int)((T.depth + kTileK - 1) / kTileK);
      if (blocks == 0) continue;
      const int n16 = round16(T.n);
      const uint32_t idesc = (1u << 4) | kind | (kAcross ? 1u << 15 : 0u) |
                             (kWeight ? 1u << 16 : 0u) | ((uint32_t)(n16 >> 3) << 17) |
                             ((uint32_t)(kTileM >> 4) << 24);
      const int buf = acc & 1;
      if (acc >= 2) ok = __all_sync(0xffffffffu, wait(C.acc_empty[buf], (acc / 2 - 1) & 1));
      tc_fence_after();
      const uint32_t d = tmem + buf * kTileN;
      for (int kb = 0; ok && kb < blocks; ++kb, ++it) {
        const int s = it % kStages;
        ok = __all_sync(0xffffffffu, wait(C.full[s], (it / kStages) & 1));
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = stages + s * kStageBytes, b = a + kABytes;
        const int left = (int)(T.depth - (int64_t)kb * kTileK);
        const int steps = left >= kTileK ? kTileK / 16 : (left + 15) / 16;
        if (kTma && kWeight && left < steps * 16) {
          // the copy took rows of the next expert along: they count as zeros
          const int boxes = 2 + (n16 + 63) / 64, gap = steps * 16 - left;
          for (int i = lane; i < boxes * gap * 8; i += 32) {
            const int box = i / (gap * 8), in = i - box * (gap * 8);
            sts128(a + box * kBoxBytes + left * 128 + in * 16, make_uint4(0, 0, 0, 0));
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) {
          const uint64_t da = kAcross ? desc_mn_sw128(a) : smem_desc_sw128(a);
          const uint64_t db = kWeight ? desc_mn_sw128(b) : smem_desc_sw128(b);
          // 16 k: 32 bytes of a row, or 16 rows
          for (int i = 0; i < steps; ++i)
            mma_f16(d, da + i * (kAcross ? 128 : 2), db + i * (kWeight ? 128 : 2), idesc,
                    kb > 0 || i > 0);
          mma_commit(smem_u32(&C.empty[s]));
          if (kb == blocks - 1) mma_commit(smem_u32(&C.acc_full[buf]));
        }
        __syncwarp();
      }
      ++acc;
    }
    if (!ok) {
      const int none = 0;
      if (lane == 0) mma_commit(smem_u32(&C.drain));
      __syncwarp();
      mbar_wait(smem_u32(&C.drain), 0, &none, kProductWaitNs / 4);
    }
  } else if (warp >= 4 && warp < 8) {
    // ---- epilogue: lane 32 * w + lane of the tile
    const int w = warp - 4;
    uint32_t acc = 0;
    bool ok = true;
    float* mine = exchange + w * 16 * 32;
    const float* other = exchange + (w ^ 2) * 16 * 32;
    for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const ProductTile T = tile_at<kMode>(A, cum, t);
      const int buf = acc & 1;
      const bool any = T.depth > 0;
      if (any) {
        // g's and u's warps go on together, or both leave
        ok = wait(C.acc_full[buf], (acc / 2) & 1);
        ok = A.gated ? barrier_all(1 + (w & 1), 64, ok) : __all_sync(0xffffffffu, ok);
      }
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(w * 32) << 16) + buf * kTileN;
      const int m = T.m0 + w * 32 + lane;
      for (int c = 0; c < T.n; c += 32) {
        uint32_t v[32];
        if (any) {
          tmem_ld32(d + c, v);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0;
        }
        const int cols = T.n - c < 32 ? T.n - c : 32;
        if (!A.gated) {
          if (m < A.M) {
            int64_t at = kWeight ? ((int64_t)T.expert * A.N + T.n0 + c) * A.M + m
                                 : (T.n0 + c) * A.M + m;
#pragma unroll
            for (int i = 0; i < 32; ++i, at += A.M)
              if (i < cols) store_value(A.out, at, __uint_as_float(v[i]), A.out_f32, A.f16);
          }
        } else if constexpr (!kWeight) {
          const int f = T.m0 + (w & 1) * 32 + lane;
          if (A.saved != nullptr && f < A.M) {
            int64_t at = (T.n0 + c) * (2 * (int64_t)A.M) + (w < 2 ? f : A.M + f);
#pragma unroll
            for (int i = 0; i < 32; ++i, at += 2 * (int64_t)A.M)
              if (i < cols) store_value(A.saved, at, __uint_as_float(v[i]), false, A.f16);
          }
          // g's warps give their upper 16 columns to u's, and get the lower ones of u
          named_bar_sync(1 + (w & 1), 64);
#pragma unroll
          for (int i = 0; i < 16; ++i) mine[i * 32 + lane] = __uint_as_float(w < 2 ? v[16 + i] : v[i]);
          named_bar_sync(1 + (w & 1), 64);
          int64_t at = (T.n0 + c + (w < 2 ? 0 : 16)) * A.M + f;
#pragma unroll
          for (int i = 0; i < 16; ++i, at += A.M) {
            const float o = other[i * 32 + lane];
            const float h = w < 2 ? silu(__uint_as_float(v[i])) * o
                                  : silu(o) * __uint_as_float(v[16 + i]);
            if (i + (w < 2 ? 0 : 16) < cols && f < A.M) store_value(A.out, at, h, false, A.f16);
          }
        }
      }
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&C.acc_empty[buf]));
        ++acc;
      }
    }
  }
  // rows that no expert has
  if (!kWeight) {
    const int64_t end = clamp_offset(A.offsets[A.E], A.R);
    const int64_t from = (int64_t)blockIdx.x * blockDim.x + tid, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = end * A.M + from; i < A.R * A.M; i += step)
      static_cast<uint16_t*>(A.out)[i] = 0;
    if (A.saved != nullptr)
      for (int64_t i = end * 2 * A.M + from; i < A.R * 2 * A.M; i += step)
        static_cast<uint16_t*>(A.saved)[i] = 0;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
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

inline hcmix_status device_sms(int* sms) {
  int dev = 0;
  const hcmix_status st = checked(cudaGetDevice(&dev));
  if (st != HCMIX_OK) return st;
  return checked(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
}

template <bool kTma, ProductMode kMode>
hcmix_status launch_product(const ProductArgs& A, int64_t most_tiles, cudaStream_t stream) {
  int sms = 0;
  const hcmix_status st = device_sms(&sms);
  if (st != HCMIX_OK) return st;
  const int64_t grid = most_tiles < sms ? (most_tiles > 0 ? most_tiles : 1) : sms;
  return launch(hcmix_product_kernel<kTma, kMode>, dim3((unsigned)grid),
                dim3(kProductThreads<kTma>), product_smem(A.E), product_smem(kProductExperts),
                stream, A);
}

// a, b, offsets, R, E, M, N, K, gated, out, saved and types are set.
template <ProductMode kMode>
hcmix_status run_product(ProductArgs& A, cudaStream_t stream) {
  constexpr bool kWeight = kMode == ProductMode::kWeight;
  const int width = A.gated ? kTileM / 2 : kTileM;
  const int64_t mt = (A.M + width - 1) / width;
  const int64_t tiles = kWeight ? A.E * mt * ((A.N + kTileN - 1) / kTileN)
                                : mt * (A.R / kTileN + (A.R < A.E ? A.R : A.E));
  const int a_experts = kWeight ? 0 : A.E;  // 0: a matrix of two dimensions
  // a box starts on 16 bytes: u's features, too, where they lie along the rows
  const bool starts = kMode != ProductMode::kRowsM || !A.gated || A.M % 8 == 0;
  if (A.R > 0 && starts && tma_readable(A.a, a_experts) && tma_readable(A.b, 0) &&
      make_box_map(&A.a_map, A.a, a_experts, A.f16, 64) &&
      make_box_map(&A.b_map, A.b, 0, A.f16, 64) && make_box_map(&A.b16_map, A.b, 0, A.f16, 16))
    return launch_product<true, kMode>(A, tiles, stream);
  return launch_product<false, kMode>(A, tiles, stream);
}

}  // namespace sublayer
}  // namespace hcmix
