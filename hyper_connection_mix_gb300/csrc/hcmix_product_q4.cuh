// Products of few rows with experts' weights of 4 bits: w = (code - 8) scale, a scale for
// each group of 32 to 256 along k.  Bound by reading the codes of the experts that have rows.
//
// A block of eight warps takes units of 32 features (16 of g and the same 16 of u where the
// product is gated) and 8 kTiles rows, one after the other from a range of its own; its warps
// share out a unit's k in chunks of 128, and add their sums in shared memory.  Codes come ahead
// through a ring of chunks of each warp's own (cp.async), without regard to the units' ends.
//
// The products are mma.m16n8k16, features as M.  The order of k within a tile is free as long
// as both operands have it: a lane's word of 8 codes of one feature, k = 8 t .. 8 t + 7 of a
// block of 32, gives its registers of two tiles, and one 16-byte load of a row the same k.  A
// code's bits under 128's (bf16) or 1024's (fp16) exponent are 128 + code, and less 136 they are
// code - 8, exactly.  Sums of a group are fp32, and are scaled and added in fp32.
//
// Meant for up to eight rows an expert: a block of rows unpacks the weights anew, so that from
// nine on the 16-bit product is faster (64 experts 5120 -> 2048 bf16, 4 and 16 bits: of 8 rows 125
// and 211 us, of 9 243 and 211, of 32 287 and 216, of 64 568 and 223), but for one expert of few
// (5120 -> 8192: 32 rows 24 and 28, 256 rows 147 and 33).
//
// Measured: 16 tokens to 8 of 128 experts 5120 -> 2 x 2048 bf16 293 us (3.1 TB/s, 45 % of the copy
// rate), one token 2048 -> 5120 fp16 27.3 us.  The copies alone take 163 us: what bounds it is
// instructions (571 of a warp for 2 KB of codes when it took 314 us).  Three blocks a
// multiprocessor with one set of registers for the rows did better than two with two sets (314 and
// 326 us); 64 features a unit did worse.
#pragma once

#include "hcmix_gate.cuh"
#include "hcmix_vec.cuh"

namespace hcmix {
namespace sublayer {

struct Q4Args {
  const void* xs;
  int64_t xs_stride, R;
  const uint8_t* codes;  // [E, N, K / 2], the lower half of a byte is the even k
  const void* scales;    // [E, N, K / group]
  const int32_t* offsets;
  int E, K, N, group;
  int gated;  // features N / 2 .. N - 1 are u's
  void* out;  // [R, N], or [R, N / 2]
  int vec;    // rows of xs start on 16 bytes
};

// (w & mask) | base in one operation, which takes one of the two from a register.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t base) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(base));
  return r;
}
__device__ __forceinline__ uint32_t q4_constant(uint32_t v) {
  uint32_t r;
  asm volatile("mov.u32 %0, %1;" : "=r"(r) : "r"(v));  // a register, whatever is known of it
  return r;
}

template <typename T>
struct Codes;
template <>
struct Codes<__nv_bfloat16> {
  uint32_t mask = q4_constant(0x000F000Fu), base = q4_constant(0x43004300u);
  uint32_t one = q4_constant(0x3F803F80u), less = q4_constant(0xC308C308u);  // 1, -136
  // codes i and i + 4 of a word, less 8 (by an fma: pairs of bf16 have no sum of their own)
  __device__ __forceinline__ uint32_t pair(uint32_t w, int i) const {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;"
        : "=r"(r)
        : "r"(and_or(w >> 4 * i, mask, base)), "r"(one), "r"(less));
    return r;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Codes<__half> {
  uint32_t even = q4_constant(0x000F000Fu), odd = q4_constant(0x00F000F0u);
  uint32_t base = q4_constant(0x64006400u), over = q4_constant(0x2C002C00u);
  uint32_t one = q4_constant(0x3C003C00u), less = q4_constant(0xE408E408u);  // 1, -1032
  uint32_t less_odd = q4_constant(0xD480D480u);                              // -72
  // the odd i need no shift: 1024 + 16 code, over 16 and less 72
  __device__ __forceinline__ uint32_t pair(uint32_t w, int i) const {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;"
        : "=r"(r)
        : "r"(and_or(i < 2 ? w : w >> 8, i % 2 ? odd : even, base)), "r"(i % 2 ? over : one),
          "r"(i % 2 ? less_odd : less));
    return r;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

constexpr int kQ4Warps = 8, kQ4Chunk = 128, kQ4Depth = 3;
constexpr int kQ4Box = 32 * kQ4Chunk / 2;  // bytes of a chunk: 32 features

// A unit's place: experts in turn, blocks of their rows in turn, features in turn.
struct Q4Place {
  int e, row, end, f;  // the expert, the block's first row, the expert's last + 1, the feature
};

__device__ __forceinline__ int q4_offset(int v, int64_t R) {
  return v < 0 ? 0 : v > R ? (int)R : v;
}

template <int kRows>
struct Q4Plan {
  const Q4Args& A;
  int features;  // outputs
  int per;       // of a unit
  int across;    // units side by side

  __device__ __forceinline__ Q4Plan(const Q4Args& a)
      : A(a), features(a.gated ? a.N / 2 : a.N), per(a.gated ? 16 : 32) {
    across = (features + per - 1) / per;
  }
  __device__ __forceinline__ int blocks(int e) const {
    const int first = q4_offset(A.offsets[e], A.R), last = q4_offset(A.offsets[e + 1], A.R);
    return last > first ? (last - first + kRows - 1) / kRows : 0;
  }
  // The first block of rows of expert e, or of the next one that has rows.
  __device__ __forceinline__ void enter(Q4Place& p, int e) const {
    for (p.e = e; p.e < A.E; ++p.e) {
      p.row = q4_offset(A.offsets[p.e], A.R);
      p.end = q4_offset(A.offsets[p.e + 1], A.R);
      if (p.end > p.row) break;
    }
    p.f = 0;
  }
  __device__ __forceinline__ void next(Q4Place& p) const {
    p.f += per;
    if (p.f < features) return;
    p.f = 0;
    p.row += kRows;
    if (p.row >= p.end) enter(p, p.e + 1);
  }
};

template <typename T, int kTiles>
struct Q4Operands {  // of a chunk: rows' k and features' scales, as a lane holds them
  uint4 x[kTiles][4];
  T scale[4];  // rows g and g + 8 of both tiles of features, block t's
};

template <typename T, int kTiles, bool kGated>
__global__ void __launch_bounds__(kQ4Warps * 32, kTiles == 1 ? 3 : 1)
    hcmix_product_q4_kernel(const Q4Args A) {
  begin_kernel();
  constexpr int kRows = 8 * kTiles;
  extern __shared__ __align__(16) uint8_t q4_shared[];
  __shared__ int64_t sums[kQ4Warps];
  __shared__ int start_of[4];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const uint32_t ring =
      (uint32_t)__cvta_generic_to_shared(q4_shared) + warp * (kQ4Depth * kQ4Box);
  float* parts = reinterpret_cast<float*>(q4_shared + kQ4Warps * kQ4Depth * kQ4Box);
  const Q4Plan<kRows> plan(A);

  // ---- the block's range of units, and the place where it begins
  const int each = (A.E + kQ4Warps * 32 - 1) / (kQ4Warps * 32);
  const int e0 = tid * each < A.E ? tid * each : A.E, e1 = e0 + each < A.E ? e0 + each : A.E;
  // (64 bits: offsets that fall may count rows many times over)
  int64_t here = 0;
  for (int e = e0; e < e1; ++e) here += plan.blocks(e);
  int64_t upto = here;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t s = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += s;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int64_t all = 0;
  for (int w = 0; w < kQ4Warps; ++w) {
    if (w < warp) upto += sums[w];
    all += sums[w];
  }
  const int64_t units = all * plan.across, per_block = units / gridDim.x;
  const int more = (int)(units % gridDim.x);
  const int64_t u0 = per_block * blockIdx.x + (blockIdx.x < more ? blockIdx.x : more);
  const int64_t u1 = u0 + per_block + (blockIdx.x < more);
  const int64_t block0 = u0 / plan.across;
  if (u0 < u1 && block0 >= upto - here && block0 < upto) {
    int64_t left = block0 - (upto - here);
    int e = e0;
    for (; left >= plan.blocks(e); ++e) left -= plan.blocks(e);
    start_of[0] = e;
    start_of[1] = q4_offset(A.offsets[e], A.R) + (int)left * kRows;
    start_of[2] = q4_offset(A.offsets[e + 1], A.R);
    start_of[3] = (int)(u0 - block0 * plan.across) * plan.per;
  }
  __syncthreads();
  const int chunks = (A.K + kQ4Chunk - 1) / kQ4Chunk;
  const int turns = (chunks + kQ4Warps - 1) / kQ4Warps;  // of a warp at a unit
  // results of more than 2^31 units a block would not fit any memory
  const int own = u1 - u0 < 0x7fffffff ? (int)(u1 - u0) : 0x7fffffff;
  const int shift = 31 - __clz(A.group), groups = A.K >> shift;
  const T* scales = static_cast<const T*>(A.scales);
  const Codes<T> code;

  if (own > 0) {
    const Q4Place start = {start_of[0], start_of[1], start_of[2], start_of[3]};
    // Feature r of a unit's 32 among its expert's, clamped to those that there are.
    const int most = plan.features - 1;
    const auto feature = [&](int f, int r) {
      const int in = f + (kGated ? r % 16 : r);
      return (in < most ? in : most) + (kGated && r >= 16 ? plan.features : 0);
    };
    // ---- codes of one chunk into a box of the ring: feature r's 64 bytes are four blocks of
    // 16, exchanged so that eight features' words of a block lie in different banks
    Q4Place ahead = start;
    int ahead_turn = 0, slot = 0;
    int ahead_left = own;
    const uint32_t to = ring + g * 64 + ((t ^ (g >> 1 & 3)) << 4);
    const uint32_t code_row = A.K / 2;
    const uint8_t* codes = nullptr;  // of ahead's expert, the lane's 16 bytes of a chunk
    uint32_t ahead_feature[4];       // the lane's
    const auto send = [&]() {
      if (ahead_left > 0) {
        if (ahead_turn == 0) {
          codes = A.codes + 16 * t + (int64_t)ahead.e * A.N * code_row;
#pragma unroll
          for (int i = 0; i < 4; ++i) ahead_feature[i] = feature(ahead.f, 8 * i + g);
          // the unit's scales will be asked for when they are needed: they are on their way to L2
          // by then.  32 (16 and 16) neighbouring features' lie side by side.
#pragma unroll
          for (int h = 0; h < (kGated ? 2 : 1); ++h) {
            const int f0 = feature(ahead.f, 16 * h), f1 = feature(ahead.f, 16 * h + plan.per - 1);
            const T* from = scales + ((int64_t)ahead.e * A.N + f0) * groups;
            const int n = (f1 - f0 + 1) * groups;
            for (int i = tid * 64; i < n; i += kQ4Warps * 32 * 64)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(from + i));
          }
        }
        const int k = (warp + ahead_turn * kQ4Warps) * kQ4Chunk;
        if (k + 32 * t < A.K) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(
                             to + slot * kQ4Box + i * 512),
                         "l"(codes + k / 2 + (uint64_t)ahead_feature[i] * code_row)
                         : "memory");
        }
        if (++slot == kQ4Depth) slot = 0;
        if (++ahead_turn == turns) {
          ahead_turn = 0;
          --ahead_left;
          plan.next(ahead);
        }
      }
      async_commit();
    };
    // ---- rows and scales of one chunk into registers
    Q4Place near = start;
    int near_turn = 0;
    int near_left = own;
    const T* of_expert = nullptr;   // scales
    uint32_t near_feature[4];       // the lane's
    const T* of_row[kTiles] = {};   // the lane's rows; behind the last the last one's again, whose
                                    // products are not stored
    const auto load = [&](Q4Operands<T, kTiles>& o) {
      if (near_left <= 0) return;
      if (near_turn == 0) {
        of_expert = scales + (int64_t)near.e * A.N * groups;
#pragma unroll
        for (int i = 0; i < 4; ++i) near_feature[i] = feature(near.f, 8 * i + g);
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          const int row = near.row + 8 * n + g;
          of_row[n] = static_cast<const T*>(A.xs) +
                      (row < near.end ? row : near.end - 1) * A.xs_stride + 8 * t;
        }
      }
      const int k = (warp + near_turn * kQ4Warps) * kQ4Chunk;
      if (A.vec && k + kQ4Chunk <= A.K) {
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int b = 0; b < 4; ++b)
            o.x[n][b] = *reinterpret_cast<const uint4*>(of_row[n] + k + 32 * b);
      } else {
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            if (k + 32 * b >= A.K) break;
            const uint16_t* p = reinterpret_cast<const uint16_t*>(of_row[n] + k + 32 * b);
            uint4& v = o.x[n][b];
            v.x = p[0] | (uint32_t)p[1] << 16, v.y = p[2] | (uint32_t)p[3] << 16;
            v.z = p[4] | (uint32_t)p[5] << 16, v.w = p[6] | (uint32_t)p[7] << 16;
          }
      }
      int q = (k + 32 * t) >> shift;
      q = q < groups ? q : groups - 1;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o.scale[i] = (of_expert + q)[(uint64_t)near_feature[i] * (uint32_t)groups];
      if (++near_turn == turns) {
        near_turn = 0;
        --near_left;
        plan.next(near);
      }
    };

    Q4Operands<T, kTiles> now;
    for (int i = 0; i < kQ4Depth - 1; ++i) send();
    Q4Place at = start;
// the blocks of a chunk with which a group (or the chunk) ends; k ends with a group
    const int ends = A.group == 32 ? 15 : A.group == 64 ? 10 : 8;
    float total[2][kTiles][4];
    int turn = 0, buf = 0, from = 0;
    const uint32_t words = ring + g * 64 + 4 * t;
    for (int left = own; left > 0;) {
      send();
      if (turn == 0) {
#pragma unroll
        for (int i = 0; i < 2 * kTiles * 4; ++i) (&total[0][0][0])[i] = 0.0f;
      }
      load(now);
      async_wait<kQ4Depth - 1>();
      __syncwarp();
      const int k = (warp + turn * kQ4Warps) * kQ4Chunk;
      const uint32_t box = words + from * kQ4Box;
      if (++from == kQ4Depth) from = 0;
      float acc[2][kTiles][4] = {};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (k + 32 * b >= A.K) break;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("ld.shared.u32 %0, [%1];"
                       : "=r"(w[i])
                       : "r"(box + i * 512 + ((b ^ (g >> 1 & 3)) << 4))
                       : "memory");
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            a[h][0] = code.pair(w[2 * h], 2 * s), a[h][1] = code.pair(w[2 * h + 1], 2 * s);
            a[h][2] = code.pair(w[2 * h], 2 * s + 1);
            a[h][3] = code.pair(w[2 * h + 1], 2 * s + 1);
          }
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            const uint4& x = now.x[n][b];
            const uint32_t lo = s ? x.y : x.x, hi = s ? x.w : x.z;
            const uint32_t b0 = __byte_perm(lo, hi, 0x5410), b1 = __byte_perm(lo, hi, 0x7632);
#pragma unroll
            for (int h = 0; h < 2; ++h) Codes<T>::mma(acc[h][n], a[h], b0, b1);
          }
        }
        if (ends >> b & 1) {
          // a group ends, or the chunk
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float s =
                  __shfl_sync(0xffffffffu, to_f32(now.scale[2 * h + i]), (lane & ~3) | b);
#pragma unroll
              for (int n = 0; n < kTiles; ++n) {
                total[h][n][2 * i] = fmaf(s, acc[h][n][2 * i], total[h][n][2 * i]);
                total[h][n][2 * i + 1] = fmaf(s, acc[h][n][2 * i + 1], total[h][n][2 * i + 1]);
                acc[h][n][2 * i] = acc[h][n][2 * i + 1] = 0.0f;
              }
            }
        }
      }
      __syncwarp();
      if (++turn < turns) continue;
      turn = 0;
      --left;
      // ---- the warps' sums: value v = (h, n, i) of a lane
      constexpr int kValues = 2 * kTiles * 4;
      float* part = parts + buf * (kQ4Warps * kValues * 32);
      buf ^= 1;  // the next unit's, which no thread writes before all have passed the barrier
#pragma unroll
      for (int v = 0; v < kValues; ++v)
        part[(warp * kValues + v) * 32 + lane] = (&total[0][0][0])[v];
      __syncthreads();
      constexpr int kOut = kGated ? kValues / 2 : kValues;
      for (int o = tid; o < kOut * 32; o += kQ4Warps * 32) {
        const int v = o / 32, h = v / (4 * kTiles), n = v / 4 % kTiles, i = v % 4;
        const auto sum = [&](int of) {
          float s = 0.0f;
#pragma unroll
          for (int w = 0; w < kQ4Warps; ++w) s += part[(w * kValues + of) * 32 + lane];
          return s;
        };
        // feature g + 8 (i / 2) of the tile, row 2 t + i % 2
        const int f = at.f + (kGated ? 0 : 16 * h) + g + 8 * (i / 2);
        const int row = at.row + 8 * n + 2 * t + i % 2;
        float y = sum(v);
        if (kGated) y = gate(y, sum(v + 4 * kTiles));
        if (f < plan.features && row < at.end)
          static_cast<T*>(A.out)[(int64_t)row * plan.features + f] = from_f32<T>(y);
      }
      plan.next(at);
    }
  }
  // rows that no expert has
  const int64_t end = q4_offset(A.offsets[A.E], A.R), step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = end * plan.features + (int64_t)blockIdx.x * blockDim.x + tid;
       i < A.R * plan.features; i += step)
    static_cast<T*>(A.out)[i] = from_f32<T>(0.0f);
}

template <int kTiles>
constexpr size_t kQ4Smem = kQ4Warps * kQ4Depth * kQ4Box + 2 * kQ4Warps * (8 * kTiles) * 32 * 4;

template <typename T, int kTiles>
hcmix_status launch_product_q4(const Q4Args& A, int sms, cudaStream_t stream) {
  const int64_t features = A.gated ? A.N / 2 : A.N, per = A.gated ? 16 : 32;
  // no more blocks than units: row blocks are at most the rows
  const int64_t most = (features + per - 1) / per * A.R;
  const int64_t grid = (int64_t)sms * (kTiles == 1 ? 3 : 1);
  const dim3 blocks((unsigned)(most < grid ? most : grid));
  const auto go = [&](auto kernel) {
    return launch(kernel, blocks, dim3(kQ4Warps * 32), kQ4Smem<kTiles>, kQ4Smem<kTiles>, stream, A);
  };
  return A.gated ? go(hcmix_product_q4_kernel<T, kTiles, true>)
                 : go(hcmix_product_q4_kernel<T, kTiles, false>);
}

inline hcmix_status run_product_q4(const Q4Args& A, hcmix_type type, cudaStream_t stream) {
  int dev = 0, sms = 0;
  hcmix_status st = checked(cudaGetDevice(&dev));
  if (st == HCMIX_OK)
    st = checked(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  if (st != HCMIX_OK) return st;
  // rows of an expert, were they shared out evenly.  One tile of 8 rows or four, measured 5120 ->
  // 8192: 8 rows 18 and 22 us, 9 rows 28 and 22, 64 rows 73 and 47; 64 experts 5120 -> 2048: of 6
  // rows 131 and 260 us, of 9 256 and 261, of 32 509 and 306.
  const bool few = A.R <= 8 * (A.R < A.E ? A.R : (int64_t)A.E);
  const auto go = [&](auto z) {
    using T = decltype(z);
    return few ? launch_product_q4<T, 1>(A, sms, stream) : launch_product_q4<T, 4>(A, sms, stream);
  };
  return type == HCMIX_BF16 ? go(__nv_bfloat16{}) : go(__half{});
}

}  // namespace sublayer
}  // namespace hcmix
