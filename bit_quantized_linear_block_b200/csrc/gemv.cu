// The quantized linear layer for few rows (1 to 16) on NVFP4 weights, and the
// same product grouped by expert when the experts have few rows each.
//
//   Y[m, n] = bf16(alpha_m sum_k a[m, k] (e2m1[n, k] * e4m3[n, k / 16]))
//
// a: integer codes (int8 or their f16 values), or bf16 rows, rotated here by
// blockdiag(H_128) when the weights are.  alpha_m = RN(g_w alpha_mul), times
// the row's scale for codes.
//
// Bound: the weights, 9/16 byte each, are read once and the rows are few, so
// HBM (L2 for a layer that stays there) is the limit and the multiply only
// has to keep up.  A 128-row tensor-memory tile would leave most of its
// columns empty and pay the pipeline's fill for one K sweep; here a warp
// streams its share of the weights straight into mma.sync fragments:
//
//   * unit: 64 weight rows (four 16-row MMA tiles) x one 128-element K block,
//     9 half-KB pieces; the rows are 16 consecutive r % 32 of one 128-row
//     scale atom and their three 32-row shifts, so that one 16-byte load of
//     scales serves the four tiles;
//   * a CTA (4 to 8 warps) owns 64 rows, its warps the K blocks of its K range
//     in turn; a cluster of S CTAs splits K further where that fills the GPU
//     more evenly.  Partial sums are added in a fixed order (warps through
//     shared memory, CTAs through distributed shared memory), so results do
//     not depend on timing and need no workspace;
//   * each lane copies the pieces it will read itself (cp.async, kGvDepth
//     blocks ahead), so the ring needs no barrier.
//
// MMA operands are f16: a weight value E2M1 x E4M3 (at most 6 significant
// bits, 2^-10 .. 2688) and an integer code are exact, products and sums are
// fp32.  A bf16 row block (rotated or not) is scaled by a power of two that
// brings its largest magnitude into [2^14, 2^15); the block's sums are scaled
// back in fp32.  Unrotated bf16 values are exact in f16 down to 2^-29 of the
// block's largest.  Rotated ones are fp32 sums and take two f16 terms, the
// value's rounding and the rounding of what is left, each with an MMA of its
// own on the same widened weights: half a step of the second term is 2^-23 of
// the value (2^-39 of the block's largest where that term is a subnormal f16).
// One term would be off by up to 2^-11 of each value, and rows whose products
// cancel would lose their result.
//
// A single row would fill one of the MMA's eight columns.  Its form lets
// column c take scale block c's elements, so a block's eight sums come out
// unscaled and are scaled in fp32: four products a tile and lane instead of 32
// f16 pairs of weights.
//
// Measured (B200, weights from HBM): 1 x 15360 x 5120 bf16 rows 12.6 us (3.5
// TB/s of weights; a copy's rate would be 6.9 us), 8 rows 17.9, 16 rows 24.7;
// to be rotated, in two terms: 14.8, 21.6, 32.9 (one term: 12.7, 18.6, 27.4);
// 16 rows of f16 codes 20.5; 5 x 5120 x 13824 int8 13.9 us; 1 x 1920 x 1920 4.1 us.
// About 3.5 us of each is launch, first loads and the sums.  What is left bounds
// differently: a single unrotated row takes 114 ns for each K block of the
// fullest SM, against 106 at an SM's share of the copy rate, but 240 units on 148
// SMs give that SM 80 K blocks where 64.9 is the average; 9 to 16 rows of codes
// take 200 ns a block for the widening's issue and latencies, with 8 to 16 warps
// on an SM by registers and shared memory (issue slots 33% active; two terms of 16
// rows: 38%, tensor pipe 37%, fixed latencies the top stall).
#include <atomic>
#include <type_traits>

#include "ql_common.cuh"
#include "gemm_common.cuh"
#include "launchers.h"
#include "segments.cuh"

namespace ql {

namespace {

constexpr int kGvRows = 64;                 // weight rows per CTA
constexpr int kGvMaxWarps = 8;
constexpr int kGvDepth = 2;                 // K blocks in flight per warp
constexpr int kGvCodeBytes = 8 * 512;       // 4 MMA tiles x 2 row halves x 32 lanes x 16 bytes
constexpr int kGvStage = kGvCodeBytes + 2 * 512;   // + the scales of both row halves
constexpr int kGvMaxCluster = 8;

enum GvAct { kGvBf16 = 0, kGvF16 = 1, kGvI8 = 2, kGvRotated = 3 };   // kGvRotated: bf16 rows to be rotated
constexpr bool gv_scaled(int act) { return act == kGvBf16 || act == kGvRotated; }   // a factor per row and K block
constexpr int gv_terms(int act) { return act == kGvRotated ? 2 : 1; }               // f16 terms of a value

// Rows of `a` as f16: 16-byte piece p = 4 row + t of plane q holds elements 32 t
// + 8 q .. + 7 of a row of the tile; the planes of the second terms follow those
// of all tiles' first.  bf16 rows come out of their rotation two to a lane, and
// 32 bytes between the pairs of rows keep its stores free of bank conflicts.
constexpr int gv_x_plane(int act) { return 512 + (gv_scaled(act) ? 128 : 0); }
constexpr int gv_x_bytes(int nt, int act) {
  return nt * (gv_terms(act) * 4 * gv_x_plane(act) + 32) + 16 + (gv_scaled(act) ? 512 : 0);
}

struct GvArgs {
  const uint8_t* a;          // rows [rows_a, K]
  const float* a_scales;     // fp32 [rows_a] (codes)
  const uint8_t* codes;      // [N, K/2], of expert e at + e * expert_codes
  const uint8_t* sf;         // MMA layout, of expert e at + e * expert_sf
  const float* gscale;       // [E]
  __nv_bfloat16* y;          // [rows, N]
  const int32_t* offsets;    // grouped: [E + 1]
  const int32_t* rows;       // grouped: source row of each output row, or null
  int64_t rows_a, rows_y;
  size_t expert_codes, expert_sf;
  int32_t M, N, K, E;
  int32_t cluster, units;
  float alpha_mul;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// The two halves of cluster_sync().
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// D (16 x 8, fp32) += A (16 x 16, f16) B (16 x 8, f16)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// As mma_f16 with a zero accumulator.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// D = A (16 x 16, bf16) B (16 x 8, bf16)
__device__ __forceinline__ void mma_bf16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t v) { return __half22float2(e4m3x2_to_f16(v)); }
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// int8 x4 -> two f16x2 words of the exact values (a byte permute builds
// 1024 + (q + 128) in f16, a packed subtract removes the offset).
__device__ __forceinline__ void i8x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 off = bits_h2(0x64806480u);   // 1152
  lo = h2_bits(__hsub2(bits_h2(__byte_perm(u, 0x64646464u, 0x4140u)), off));
  hi = h2_bits(__hsub2(bits_h2(__byte_perm(u, 0x64646464u, 0x4342u)), off));
}

// This lane's 32 codes [32 t, 32 t + 32) of a 128-element block as 16 f16x2
// words, t = lane % 4.
template <int ACT>
__device__ __forceinline__ void codes_to_f16(const uint4 (&raw)[4], uint32_t (&w)[16]) {
  if constexpr (ACT == kGvF16) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      w[4 * q] = raw[q].x;
      w[4 * q + 1] = raw[q].y;
      w[4 * q + 2] = raw[q].z;
      w[4 * q + 3] = raw[q].w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      i8x4_to_f16x4(raw[q].x, w[8 * q], w[8 * q + 1]);
      i8x4_to_f16x4(raw[q].y, w[8 * q + 2], w[8 * q + 3]);
      i8x4_to_f16x4(raw[q].z, w[8 * q + 4], w[8 * q + 5]);
      i8x4_to_f16x4(raw[q].w, w[8 * q + 6], w[8 * q + 7]);
    }
  }
}

// The rotation of bf16 rows.  H_128 is H_16 over four bits of the element index
// times H_8 over the other three.  Bits 0, 2, 5, 6 are one MMA's k index as the
// rows lie in the lanes (k = 2 t + i0 + 8 i2: bits 5 and 6 are t, 0 and 2 the
// place in a loaded 16-byte piece), so eight MMAs with +-1 do H_16 without an
// exchange of lanes or an unpacked value, and leave the eight values of bits 1,
// 3, 4 in one lane, two rows at a time, for packed butterflies.  8 MMAs and 48
// packed operations for 8 rows in place of 128 and 64 lane exchanges: with one
// term to a value, 8 x 15360 x 5120 took 18.4 us against 20.8, 16 rows 27.5
// against 33.0.  Products are exact, sums fp32.  Without a rotation A is the
// matching permutation.
template <int ACT>
__device__ __forceinline__ void rotation_operand(uint32_t (&a)[4]) {
  const int lane = static_cast<int>(lane_id()), g = lane >> 2, t = lane & 3;
  const uint32_t s = ((g >> 1) & t & 1) ^ ((g >> 2) & (t >> 1) & 1);   // sign of bits 5 and 6
  const uint32_t s2 = s ^ (g & 1);                                     // and of bit 2
  auto pair = [](uint32_t lo, uint32_t hi) { return 0x3F803F80u ^ (lo << 15) ^ (hi << 31); };
  a[0] = pair(s, s);
  a[1] = pair(s, s ^ 1);        // row g + 8: bit 0
  a[2] = pair(s2, s2);
  a[3] = pair(s2, s2 ^ 1);
  if constexpr (ACT == kGvBf16) {
    const uint32_t here = t == (g >> 1) ? 0x3F80u : 0u;
    a[0] = (g & 1) ? 0u : here;
    a[1] = (g & 1) ? 0u : here << 16;
    a[2] = (g & 1) ? here : 0u;
    a[3] = (g & 1) ? here << 16 : 0u;
  }
}

// A K block of 8 rows, row `lane / 4` in its four lanes as loaded, rotated by
// `a` (kept in shared memory between the blocks: four registers less), each row
// scaled by its power of two and rounded to f16, into the tile's planes at
// `dst`; the second terms of rotated values `second` bytes behind; the factors
// that undo the scaling to `factor`.
template <int ACT>
__device__ __forceinline__ void rotate_block(const uint4 (&raw)[4], const uint32_t (&a)[4], uint8_t* dst, int second,
                                             float* factor) {
  const int lane = static_cast<int>(lane_id()), g = lane >> 2, t = lane & 3;
  float2 P[4][2][2];   // [bits 3, 4][bit 1][bit 0] of rows 2 t and 2 t + 1
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float d[4];
    mma_bf16_zero(d, a, raw[q].x, raw[q].z);
    P[q][0][0] = make_float2(d[0], d[1]);
    P[q][0][1] = make_float2(d[2], d[3]);
    mma_bf16_zero(d, a, raw[q].y, raw[q].w);
    P[q][1][0] = make_float2(d[0], d[1]);
    P[q][1][1] = make_float2(d[2], d[3]);
  }
  if constexpr (ACT == kGvRotated) {
    auto butterfly = [](float2& x, float2& y) {
      const float2 u = x, v = y;
      x = __fadd2_rn(u, v);
      y = __ffma2_rn(v, make_float2(-1.f, -1.f), u);
    };
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int q = 0; q < 4; ++q) butterfly(P[q][0][k], P[q][1][k]);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        butterfly(P[0][b][k], P[1][b][k]);
        butterfly(P[2][b][k], P[3][b][k]);
        butterfly(P[0][b][k], P[2][b][k]);
        butterfly(P[1][b][k], P[3][b][k]);
      }
    }
  }
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      m0 = fmax3(m0, fabsf(P[q][b][0].x), fabsf(P[q][b][1].x));
      m1 = fmax3(m1, fabsf(P[q][b][0].y), fabsf(P[q][b][1].y));
    }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
  }
  // 2^(141 - e) brings [2^(e - 127), 2^(e - 126)) to [2^14, 2^15); e >= 15
  // keeps it and its inverse normal numbers (a smaller block's values are
  // multiples of 2^-133, 2^-7 when scaled: still exact in the two terms)
  const uint32_t e0 = max(__float_as_uint(m0) >> 23, 15u), e1 = max(__float_as_uint(m1) >> 23, 15u);
  const float2 mul = make_float2(__uint_as_float((268u - e0) << 23), __uint_as_float((268u - e1) << 23));
  uint8_t* out = dst + t * 160 + (g >> 1) * 16 + (g & 1) * 8;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w0[2], w1[2], v0[2], v1[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float2 lo = __fmul2_rn(P[q][b][0], mul), hi = __fmul2_rn(P[q][b][1], mul);
      const __half2 r0 = __floats2half2_rn(lo.x, hi.x), r1 = __floats2half2_rn(lo.y, hi.y);
      w0[b] = h2_bits(r0);
      w1[b] = h2_bits(r1);
      if constexpr (ACT == kGvRotated) {   // what the first term leaves, exact in fp32
        const float2 f0 = __half22float2(r0), f1 = __half22float2(r1);
        v0[b] = h2_bits(__floats2half2_rn(lo.x - f0.x, hi.x - f0.y));
        v1[b] = h2_bits(__floats2half2_rn(lo.y - f1.x, hi.y - f1.y));
      }
    }
    *reinterpret_cast<uint2*>(out + q * gv_x_plane(ACT)) = make_uint2(w0[0], w0[1]);
    *reinterpret_cast<uint2*>(out + q * gv_x_plane(ACT) + 64) = make_uint2(w1[0], w1[1]);
    if constexpr (ACT == kGvRotated) {
      *reinterpret_cast<uint2*>(out + second + q * gv_x_plane(ACT)) = make_uint2(v0[0], v0[1]);
      *reinterpret_cast<uint2*>(out + second + q * gv_x_plane(ACT) + 64) = make_uint2(v1[0], v1[1]);
    }
  }
  if (g == 0) {
    factor[2 * t] = __uint_as_float((e0 - 14u) << 23);
    factor[2 * t + 1] = __uint_as_float((e1 - 14u) << 23);
  }
}

}  // namespace

// The threads that the compiler makes registers for: 16 warps on an SM, 12 with
// two row tiles or two terms, 8 with both (224 registers; at 12 warps it spills
// 300 bytes: 16 x 15360 x 5120 42.5 against 36.7 us).
constexpr int gv_max_threads(int nt, int act) { return (nt == 1) == (act == kGvRotated) ? 384 : 32 * kGvMaxWarps; }
constexpr int gv_min_ctas(int nt, int act) { return nt == 1 && act != kGvRotated ? 2 : 1; }

// NT: tiles of 8 rows of `a` (1: up to 8 rows, 2: up to 16).  ONE: the form
// for a single row (0 never, 1 always, 2 where a row tile has one row).
template <int NT, int ACT, bool GROUPED, int ONE>
__global__ void __launch_bounds__(gv_max_threads(NT, ACT), gv_min_ctas(NT, ACT)) k_gemv(const GvArgs p) {
  constexpr int kTokens = 8 * NT;
  constexpr bool kScaled = gv_scaled(ACT);
  constexpr int kPlane = gv_x_plane(ACT);
  constexpr int kXBytes = gv_x_bytes(NT, ACT);
  constexpr int kSecond = NT * 4 * kPlane;       // from a first term to its second
  constexpr int kXScale = gv_terms(ACT) * kSecond;
  constexpr int kXZero = kXScale + NT * 32;      // a warp's rows of `a` and their factors, 16 zero bytes, the rotation's operand
  constexpr int kRaw = ACT == kGvI8 ? 2 : 4;     // 16-byte pieces of a lane's 32 elements
  extern __shared__ __align__(16) uint8_t smem[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  const int lane = static_cast<int>(lane_id()), g = lane >> 2, t = lane & 3;
  const int S = p.cluster;
  const int block = blockIdx.x / S, rank = blockIdx.x - block * S;
  const int unit = GROUPED ? block % p.units : block;
  pdl_wait();

  int M = p.M;
  int64_t row0 = 0;
  const uint8_t* codes = p.codes;
  const uint8_t* sf = p.sf;
  const float* gscale = p.gscale;
  if constexpr (GROUPED) {
    // block / units counts the row tiles of all experts in order
    int tile = block / p.units, e0 = 0;
    bool found = false;
    int64_t carry = 0;
    for (; e0 < p.E; e0 += 32) {
      int64_t lo, hi;
      warp_segments(p.offsets, p.E, p.rows_y, e0 + lane, carry, lo, hi);
      const int cnt = static_cast<int>(hi - lo), tiles = (cnt + kTokens - 1) / kTokens;
      const int end = warp_inclusive_sum(tiles);
      const unsigned hit = __ballot_sync(0xffffffffu, tile < end);
      if (hit != 0) {
        const int src = __ffs(hit) - 1;
        const int first = __shfl_sync(0xffffffffu, end - tiles, src);
        const int c = __shfl_sync(0xffffffffu, cnt, src);
        row0 = __shfl_sync(0xffffffffu, lo, src) + static_cast<int64_t>(tile - first) * kTokens;
        M = min(kTokens, c - (tile - first) * kTokens);
        e0 += src;
        found = true;
        break;
      }
      tile -= __shfl_sync(0xffffffffu, end, 31);
    }
    if (!found) {                                // past the last tile: the same for the whole cluster
      pdl_release();
      return;
    }
    codes += static_cast<size_t>(e0) * p.expert_codes;
    sf += static_cast<size_t>(e0) * p.expert_sf;
    gscale += e0;
  }

  // 64 weight rows of this CTA: tile i holds rows first + 32 i .. + 15
  const int first = 128 * (unit >> 1) + 16 * (unit & 1);
  const int ntiles = min(4, (p.N - first + 31) / 32);          // tiles inside N (N and the tiles are 16-aligned)
  const int kb_all = p.K >> 7;
  const int kb0 = static_cast<int>(static_cast<int64_t>(kb_all) * rank / S);
  const int kb1 = static_cast<int>(static_cast<int64_t>(kb_all) * (rank + 1) / S);
  const int nblk = max(0, (kb1 - kb0 - warp + warps - 1) / warps);   // blocks kb0 + warp + j * warps
  const size_t row_bytes = static_cast<size_t>(p.K) / 2;
  const uint8_t* wsrc = codes + static_cast<size_t>(first + g) * row_bytes + 16 * t;
  const uint8_t* ssrc = sf + (static_cast<size_t>(unit >> 1) * (p.K >> 6) + (t >> 1)) * 512 +
                        static_cast<size_t>(16 * (unit & 1) + g) * 16;
  uint8_t* ring = smem + warp * (kGvDepth * kGvStage);
  uint8_t* xbuf = smem + warps * (kGvDepth * kGvStage) + warp * kXBytes;
  float* xscale = reinterpret_cast<float*>(xbuf + kXScale);
  if (lane == 0) *reinterpret_cast<uint4*>(xbuf + kXZero) = make_uint4(0, 0, 0, 0);   // read in place of rows that are not there
  // This lane's pieces of block 0, moved on by a block of this warp with each
  // issue.  Tiles past N copy tile 0 again (their sums are not stored).
  const uint8_t* wp[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    wp[i] = wsrc + static_cast<size_t>(i < ntiles ? 32 * i : 0) * row_bytes + static_cast<size_t>(kb0 + warp) * 64;
  const uint8_t* sp = ssrc + static_cast<size_t>(kb0 + warp) * 1024;
  const size_t half = 8 * row_bytes;
  auto issue = [&](int j) {                      // weights and scales of block j into its ring slot
    if (j < nblk) {
      const uint32_t dst = smem_u32(ring + (j % kGvDepth) * kGvStage) + 16 * lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cp_async16(dst + (2 * i) * 512, wp[i]);
        cp_async16(dst + (2 * i + 1) * 512, wp[i] + half);
        wp[i] += 64 * warps;
      }
      cp_async16(dst + kGvCodeBytes, sp);
      cp_async16(dst + kGvCodeBytes + 512, sp + 128);
      sp += 1024 * warps;
    }
    cp_async_commit();                           // a group per block, empty past the end
  };
#pragma unroll
  for (int j = 0; j < kGvDepth; ++j) issue(j);

  // Rows of `a`: lane group g (four lanes) converts one (block, row) pair of a
  // batch of `gb` blocks x `m2` rows, gb m2 = 8 (NT = 2: one block, 8 rows twice).
  const bool one = NT == 1 && (ONE == 1 || (ONE == 2 && M == 1));
  const int m2 = NT == 2 ? 8 : M > 4 ? 8 : M > 2 ? 4 : M;
  const int gb = 8 / m2;
  const int pair_blk = g / m2, pair_row = g - pair_blk * m2;
  const uint8_t* asrc[NT];
  bool a_ok[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int m = 8 * nt + pair_row;
    int64_t src = row0 + m;
    a_ok[nt] = m < M;
    if (GROUPED && p.rows != nullptr && a_ok[nt]) src = p.rows[row0 + m];
    a_ok[nt] = a_ok[nt] && src >= 0 && src < p.rows_a;
    asrc[nt] = p.a + (static_cast<size_t>(a_ok[nt] ? src : 0) * p.K + 32 * t) * (ACT == kGvI8 ? 1 : 2);
  }
  uint4 raw[NT][4];
  auto load_a = [&](int j0) {
    const int j = j0 + pair_blk;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint8_t* src = asrc[nt] + static_cast<size_t>(kb0 + warp + j * warps) * (ACT == kGvI8 ? 128 : 256);
#pragma unroll
      for (int q = 0; q < kRaw; ++q)
        raw[nt][q] = (a_ok[nt] && j < nblk) ? *reinterpret_cast<const uint4*>(src + 16 * q) : make_uint4(0, 0, 0, 0);
    }
  };

  float acc[4][NT][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][nt][c] = 0.f;

  if constexpr (kScaled) {
    uint32_t rot[4];
    rotation_operand<ACT>(rot);
    *reinterpret_cast<uint4*>(xbuf + kXZero + 16 + 16 * lane) = make_uint4(rot[0], rot[1], rot[2], rot[3]);
  }
  if (nblk > 0) load_a(0);
  for (int j0 = 0; j0 < nblk; j0 += gb) {
    __syncwarp();                                // the previous batch has been read
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (kScaled) {
        const uint4 r = lds128(xbuf + kXZero + 16 + 16 * lane);
        const uint32_t rot[4] = {r.x, r.y, r.z, r.w};
        rotate_block<ACT>(raw[nt], rot, xbuf + nt * 4 * kPlane, kSecond, xscale + 8 * nt);
      } else {
        uint32_t w[16];
        codes_to_f16<ACT>(raw[nt], w);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(xbuf + (4 * nt + q) * kPlane + lane * 16) =
              make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
      }
    }
    __syncwarp();
    if (j0 + gb < nblk) load_a(j0 + gb);
    const int batch = min(gb, nblk - j0);
    for (int b = 0; b < batch; ++b) {
      const int j = j0 + b;
      cp_async_wait<kGvDepth - 1>();             // this lane's own pieces of block j have landed
      const uint8_t* slot = ring + (j % kGvDepth) * kGvStage + 16 * lane;
      // B fragments: row g of the tile, elements 32 t + 8 q ..; for a single
      // row, column g takes scale block g's elements only
      auto x_piece = [&](int nt, int q, int second) {
        const bool mine = one ? g == 2 * t + (q >> 1) : g < m2;
        const int piece = one ? 4 * b + t : b * m2 * 4 + lane;
        const int at = (4 * nt + q) * kPlane + piece * 16 + (kScaled ? (piece >> 3) * 32 : 0);
        return lds128(xbuf + (mine ? at + second : kXZero));
      };
      uint4 xf[NT][4];   // two terms: loaded plane by plane, for registers
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if constexpr (ACT != kGvRotated) xf[nt][q] = x_piece(nt, q, 0);
      const uint4 sa = lds128(slot + kGvCodeBytes), sb = lds128(slot + kGvCodeBytes + 512);
      const uint32_t sa4[4] = {sa.x, sa.y, sa.z, sa.w}, sb4[4] = {sb.x, sb.y, sb.z, sb.w};
      float f0[NT], f1[NT];
      if constexpr (kScaled) {                   // factors of rows 2t and 2t + 1 (columns of the accumulator)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          f0[nt] = xscale[8 * nt + (one ? b : min(b * m2 + 2 * t, 7))];
          f1[nt] = xscale[8 * nt + min(b * m2 + 2 * t + 1, 7)];
        }
      }
      // All four tiles, step by step, so that their chains of dependent MMAs
      // overlap (a tile at a time, each waits for its own eight).  A tile past N
      // multiplies tile 0's weights again; nothing of it is stored.
      uint4 ca[4], cb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ca[i] = lds128(slot + (2 * i) * 512);
        cb[i] = lds128(slot + (2 * i + 1) * 512);
      }
      if (one) {
        // Column c of the accumulator is the sum over scale block c of the
        // unscaled values, so each lane scales its columns 2 t and 2 t + 1 in
        // fp32, four values a tile, instead of 32 f16 pairs of weights.
        float part[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 xs{};   // the second terms
          if constexpr (ACT == kGvRotated) {
            xf[0][q] = x_piece(0, q, 0);
            xs = x_piece(0, q, kSecond);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t ha[4], hb[4];
            fp4x8_to_f16(word_of(ca[i], q), ha);
            fp4x8_to_f16(word_of(cb[i], q), hb);
            if (q == 0) mma_f16_zero(part[i], ha[0], hb[0], ha[1], hb[1], xf[0][q].x, xf[0][q].y);
            else mma_f16(part[i], ha[0], hb[0], ha[1], hb[1], xf[0][q].x, xf[0][q].y);
            mma_f16(part[i], ha[2], hb[2], ha[3], hb[3], xf[0][q].z, xf[0][q].w);
            if constexpr (ACT == kGvRotated) {
              mma_f16(part[i], ha[0], hb[0], ha[1], hb[1], xs.x, xs.y);
              mma_f16(part[i], ha[2], hb[2], ha[3], hb[3], xs.z, xs.w);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 fa = e4m3x2_to_f32(sa4[i] >> (16 * (t & 1))), fb = e4m3x2_to_f32(sb4[i] >> (16 * (t & 1)));
          const float va = fmaf(part[i][1], fa.y, __fmul_rn(part[i][0], fa.x));
          const float vb = fmaf(part[i][3], fb.y, __fmul_rn(part[i][2], fb.x));
          acc[i][0][0] = kScaled ? fmaf(va, f0[0], acc[i][0][0]) : acc[i][0][0] + va;
          acc[i][0][2] = kScaled ? fmaf(vb, f0[0], acc[i][0][2]) : acc[i][0][2] + vb;
        }
        issue(j + kGvDepth);
        continue;
      }
      float part[4][NT][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint4 xs[NT];   // the second terms
        if constexpr (ACT == kGvRotated) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            xf[nt][q] = x_piece(nt, q, 0);
            xs[nt] = x_piece(nt, q, kSecond);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // scales of elements 32 t .. 32 t + 31, one per 16; this q's as an f16 pair
          const __half2 s2a = e4m3x2_to_f16(sa4[i] >> (16 * (t & 1))), s2b = e4m3x2_to_f16(sb4[i] >> (16 * (t & 1)));
          const __half2 va = q < 2 ? __low2half2(s2a) : __high2half2(s2a);
          const __half2 vb = q < 2 ? __low2half2(s2b) : __high2half2(s2b);
          uint32_t ha[4], hb[4];
          fp4x8_to_f16(word_of(ca[i], q), ha);
          fp4x8_to_f16(word_of(cb[i], q), hb);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            ha[c] = h2_bits(__hmul2(bits_h2(ha[c]), va));
            hb[c] = h2_bits(__hmul2(bits_h2(hb[c]), vb));
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float (&d)[4] = kScaled ? part[i][nt] : acc[i][nt];
            if (kScaled && q == 0) mma_f16_zero(d, ha[0], hb[0], ha[1], hb[1], xf[nt][q].x, xf[nt][q].y);
            else mma_f16(d, ha[0], hb[0], ha[1], hb[1], xf[nt][q].x, xf[nt][q].y);
            mma_f16(d, ha[2], hb[2], ha[3], hb[3], xf[nt][q].z, xf[nt][q].w);
            if constexpr (ACT == kGvRotated) {
              mma_f16(d, ha[0], hb[0], ha[1], hb[1], xs[nt].x, xs[nt].y);
              mma_f16(d, ha[2], hb[2], ha[3], hb[3], xs[nt].z, xs[nt].w);
            }
          }
        }
      }
      if constexpr (kScaled) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[i][nt][0] = fmaf(part[i][nt][0], f0[nt], acc[i][nt][0]);
            acc[i][nt][1] = fmaf(part[i][nt][1], f1[nt], acc[i][nt][1]);
            acc[i][nt][2] = fmaf(part[i][nt][2], f0[nt], acc[i][nt][2]);
            acc[i][nt][3] = fmaf(part[i][nt][3], f1[nt], acc[i][nt][3]);
          }
      }
      issue(j + kGvDepth);                       // the slot just read
    }
  }
  cp_async_wait<0>();
  __syncthreads();                               // the ring is free: it becomes the reduction buffer
  if (S > 1) cluster_arrive();

  // acc[i][nt][c]: weight row 16 i + g + 8 (c / 2) of the unit, row 8 nt + 2 t + c % 2 of a
  constexpr int kPitch = kGvRows + 1;
  float* red = reinterpret_cast<float*>(smem);   // [warps][kTokens][kPitch]
  float* parts = red + warps * kTokens * kPitch; // the cluster's first CTA: [S][kTokens][kGvRows]
  if (one) {   // a row's sum is spread over the four lanes of its scale blocks
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 4; c += 2) {
        acc[i][0][c] += __shfl_xor_sync(0xffffffffu, acc[i][0][c], 1);
        acc[i][0][c] += __shfl_xor_sync(0xffffffffu, acc[i][0][c], 2);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        red[(warp * kTokens + 8 * nt + 2 * t + (c & 1)) * kPitch + 16 * i + g + 8 * (c >> 1)] = acc[i][nt][c];
  __syncthreads();
  auto warps_sum = [&](int m, int r) {
    float v = 0.f;
    for (int w = 0; w < warps; ++w) v += red[(w * kTokens + m) * kPitch + r];
    return v;
  };
  if (S > 1) {   // the CTA's sums to the cluster's first CTA
    cluster_wait();   // every CTA of the cluster has started, and the first one's ring is free
    const uint32_t dst = map_to_rank(smem_u32(parts + rank * kTokens * kGvRows), 0);
    for (int o = threadIdx.x; o < M * kGvRows; o += blockDim.x) st_cluster_f32(dst + 4 * o, warps_sum(o >> 6, o & 63));
    __syncwarp();
    cluster_sync();
    if (rank != 0) {
      pdl_release();
      return;
    }
  }
  const float alpha = __fmul_rn(ld_dep(gscale), p.alpha_mul);
  for (int o = threadIdx.x; o < M * kGvRows; o += blockDim.x) {
    const int m = o >> 6, r = o & 63;
    const int n = first + 32 * (r >> 4) + (r & 15);
    float v = 0.f;
    if (S > 1)
      for (int c = 0; c < S; ++c) v += parts[c * kTokens * kGvRows + o];
    else
      v = warps_sum(m, r);
    if (n < p.N) {
      float a = alpha;
      if constexpr (!kScaled) {
        int64_t src = row0 + m;
        if (GROUPED && p.rows != nullptr) src = p.rows[row0 + m];
        a = src >= 0 && src < p.rows_a ? __fmul_rn(alpha, ld_dep(p.a_scales + src)) : 0.f;
      }
      p.y[(row0 + m) * p.N + n] = __float2bfloat16_rn(__fmul_rn(a, v));
    }
  }
  pdl_release();
}

namespace {

// 64-row units with at least one 16-row tile inside N.
int gemv_units(int32_t N) {
  const int r = N % 128;
  return 2 * (N / 128) + (r == 0 ? 0 : r > 16 ? 2 : 1);
}

// CTAs that a split of K over S CTAs of a cluster is reckoned to run at once, one
// to an SM; 0 for a split that is not tried.  From three CTAs on clusters do not
// fill every SM (eight warps to a CTA: 296 CTAs are resident at S = 1 and 2, 264
// to 284 at 3 to 8, but 259 at 7).  S = 7 was the best split of none of the 72
// layers and row counts where it was measured.
int64_t split_room(int S, int64_t k_blocks, int sms) {
  if (S == 7 || (S > 1 && 2 * S > k_blocks)) return 0;
  return S < 3 ? sms : sms - 8;
}

// Clusters of S CTAs of a kernel that are resident at once, -1 for none, 0 if
// that cannot be found out now.
int max_clusters(const void* kern, int S, int warps, int smem) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(S * num_sms()));
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (!set_smem_attr(kern, smem) || cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  return n > 0 ? n : -1;
}

// tiles: row tiles (grouped: the most that the experts' rows can make).
template <int NT, int ACT, bool GROUPED, int ONE>
ql_status launch_gemv_cfg(GvArgs p, int64_t tiles, cudaStream_t st) {
  const int units = gemv_units(p.N), kb = p.K / 128;
  const int64_t ctas = units * tiles;
  auto kern = k_gemv<NT, ACT, GROUPED, ONE>;
  auto smem_for = [&](int warps, int S) {
    const int ring = warps * (kGvDepth * kGvStage + gv_x_bytes(NT, ACT));
    const int red = 8 * NT * (warps * (kGvRows + 1) + (S > 1 ? S * kGvRows : 0)) * 4;
    return std::max(ring, red);
  };
  auto resident = [&](int S, int warps) {   // CTAs that run at once
    static std::atomic<int> known[kGvMaxCluster + 1][kGvMaxWarps + 1];   // the same for every device
    int n = known[S][warps].load(std::memory_order_relaxed);
    if (n == 0) {
      n = max_clusters(reinterpret_cast<const void*>(kern), S, warps, smem_for(warps, S));
      known[S][warps].store(n, std::memory_order_relaxed);   // 0: asked again by the next call
    }
    return static_cast<int64_t>(n) * S;
  };
  // K split over S CTAs of a cluster, and the warps of a CTA, by the least of an
  // estimate in ns, fitted to 108 layers and row counts at every split (its
  // choices are 1.6 to 4% behind the best ones on average, S = 1 with eight
  // warps 31%): the K blocks of the fullest SM, the turns that a warp takes, the
  // cluster's barrier and hand-over, the warps of an SM, and the sums that a
  // CTA's threads add up.  Clusters run together or not at all (2400 x 11904
  // 12.5 us at S = 7, whose 38 clusters are one too many, against 8.2 at 6); from
  // three CTAs on they do not fill every SM evenly.  Waves of single CTAs cost
  // their start again, and with 8 warps on an SM more than that (16 rows of 15360
  // x 5120 to be rotated: two waves of eight warps 36.7 us, one of four 32.8).
  // The two-term form was added later: over 18 layers at 1, 3, 8 and 16 rows its
  // choices are 1.1 to 2.4% behind.
  constexpr bool kOne = !GROUPED && ONE == 1;
  const int rows = GROUPED ? (NT == 1 ? 2 : 12) : p.M;   // of a row tile (grouped: unknown here)
  const int sms = num_sms();
  int S = 1, warps = 4;
  int64_t best = INT64_MAX;
  for (int s = 1; s <= kGvMaxCluster; ++s) {
    const int64_t room = split_room(s, kb, sms);
    if (room == 0) continue;
    const int64_t sm_ctas = (ctas * s + room - 1) / room;
    const int per_cta = (kb + s - 1) / s;
    for (int w : {4, 5, 6, 8}) {
      int64_t cost = sm_ctas * per_cta * (kOne ? 90 : NT == 1 ? 130 : 200) +
                     (per_cta + w - 1) / w * (gv_scaled(ACT) && !kOne ? 700 : 330) +
                     (s == 1 ? 0 : kOne ? 900 : 1450) + sm_ctas * w * (NT == 1 ? 130 : 220) + 700 * rows / w;
      if (cost >= best) continue;
      const int64_t run = resident(s, w);
      if (s > 1 && ctas * s > run) continue;
      if (s == 1 && run > 0) cost += (ctas - 1) / run * (NT == 2 && ACT == kGvRotated ? 6000 : 2000);
      if (cost < best) {
        best = cost;
        S = s;
        warps = w;
      }
    }
  }
  if (ctas * S > 0x7FFFFFFF) return QL_ERR_UNSUPPORTED_SHAPE;
  p.cluster = S;
  p.units = units;
  const int smem = smem_for(warps, S);
  if (!set_smem_attr(reinterpret_cast<const void*>(kern), smem)) return QL_ERR_CUDA;
  if (launch_pdl(kern, dim3(static_cast<unsigned>(ctas * S)), dim3(32 * warps), smem, st, S, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return QL_ERR_CUDA;
  }
  return QL_OK;
}

}  // namespace

ql_status launch_gemv(int act, const void* a, const float* a_scales, int64_t M, const ql_weights* w, void* Y,
                      cudaStream_t st) {
  if (M == 0) return QL_OK;
  GvArgs p{};
  p.a = static_cast<const uint8_t*>(a);
  p.a_scales = a_scales;
  p.codes = static_cast<const uint8_t*>(w->codes);
  p.sf = static_cast<const uint8_t*>(w->sf);
  p.gscale = w->gscale;
  p.y = static_cast<__nv_bfloat16*>(Y);
  p.rows_a = p.rows_y = M;
  p.M = static_cast<int32_t>(M);
  p.N = w->N;
  p.K = w->K;
  p.alpha_mul = w->hadamard ? (1.0f / 128.0f) : 1.0f;
  auto by_act = [&](auto nt, auto one) {
    constexpr int NT = decltype(nt)::value, ONE = decltype(one)::value;
    return act == 0 && w->hadamard ? launch_gemv_cfg<NT, kGvRotated, false, ONE>(p, 1, st)
           : act == 0 ? launch_gemv_cfg<NT, kGvBf16, false, ONE>(p, 1, st)
           : act == 1 ? launch_gemv_cfg<NT, kGvF16, false, ONE>(p, 1, st)
                      : launch_gemv_cfg<NT, kGvI8, false, ONE>(p, 1, st);
  };
  using std::integral_constant;
  if (M == 1) return by_act(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (M <= 8) return by_act(integral_constant<int, 1>{}, integral_constant<int, 0>{});
  return by_act(integral_constant<int, 2>{}, integral_constant<int, 0>{});
}

// Rows of a row tile: 8 unless the experts' rows fill more on average.
static int grouped_few_rows(int64_t T, int64_t E) { return T <= 8 * E ? 8 : 16; }

// ns beyond the launch: the K blocks of the fullest SM at the best split of K
// whose CTAs are resident together (16 warps an SM, 12 with 16-row tiles), each
// 150 ns, 250 with 16-row tiles, and 1 us more for those.  Chosen by this
// estimate against that of the tensor-memory tiles, 252 shapes of 1 to 512
// rows, 1 to 64 experts, 32 x 896 to 7680 x 1920, lose 0.2% to the better form on
// average (always tiles 32%, always this form 18%); us, this form / tiles: one
// expert 160 x 2816 at 256 rows 9.9 / 13.0, 1920 x 1920 at 64 rows 8.6 / 10.1 and
// at 256 22.9 / 11.6, seven 288 x 5120 at 32 rows 9.3 / 16.5.
int64_t grouped_few_ns(int64_t T, int64_t E, int64_t N, int64_t K) {
  const int rows = grouped_few_rows(T, E);
  const int64_t ctas = gemv_units(static_cast<int32_t>(N)) * most_row_tiles(T, E, rows), kb = K / 128;
  int64_t blocks = INT64_MAX;
  for (int s = 1; s <= kGvMaxCluster; ++s) {
    const int64_t room = split_room(s, kb, kEstimateSms);
    if (room == 0) continue;
    const int64_t sm_ctas = (ctas * s + room - 1) / room, per_cta = (kb + s - 1) / s;
    if (s > 1 && sm_ctas * std::max<int64_t>(4, std::min<int64_t>(kGvMaxWarps, per_cta)) > (rows == 8 ? 16 : 12)) break;
    blocks = std::min(blocks, sm_ctas * per_cta);
  }
  return rows == 8 ? 150 * blocks : 1000 + 250 * blocks;
}

ql_status launch_grouped_few(const void* a, const float* a_scales, int64_t rows_a, const int32_t* rows,
                             const int32_t* offsets, int64_t T, const ql_experts* w, void* Y, cudaStream_t st) {
  GvArgs p{};
  p.a = static_cast<const uint8_t*>(a);
  p.a_scales = a_scales;
  p.codes = static_cast<const uint8_t*>(w->codes);
  p.sf = static_cast<const uint8_t*>(w->sf);
  p.gscale = w->gscale;
  p.y = static_cast<__nv_bfloat16*>(Y);
  p.offsets = offsets;
  p.rows = rows;
  p.rows_a = rows_a;
  p.rows_y = T;
  p.expert_codes = static_cast<size_t>(w->N) * w->K / 2;
  p.expert_sf = qlinear_sf_bytes(w->N, w->K);
  p.N = w->N;
  p.K = w->K;
  p.E = w->E;
  p.alpha_mul = w->hadamard ? (1.0f / 128.0f) : 1.0f;
  return grouped_few_rows(T, w->E) == 8
             ? launch_gemv_cfg<1, kGvF16, true, 2>(p, most_row_tiles(T, w->E, 8), st)
             : launch_gemv_cfg<2, kGvF16, true, 0>(p, most_row_tiles(T, w->E, 16), st);
}

}  // namespace ql
