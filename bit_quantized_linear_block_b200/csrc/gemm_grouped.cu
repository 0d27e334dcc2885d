// The quantized linear layer grouped by expert: ragged row segments of
// f16-coded integer activations, each times its own expert's NVFP4 weights.
//
//   Y[r, n] = bf16(RN(RN(g_e alpha_mul) s[src]) * sum_k q[src, k] W_e[n, k]),
//   r in [offsets[e], offsets[e+1]), src = rows[r] (or r)
//
// Bound: the tensor cores when experts have many rows (2 T N K flop), the
// packed weights' bytes when they have few.  The weights are widened on chip:
// E2M1 x E4M3 is exact in f16, and a tcgen05.mma takes its A operand from
// tensor memory, so the kernel computes the transposed tile
// D[n, m] = sum_k W[n, k] q[m, k] (128 weight rows on the TMEM lanes, up to
// BMT rows of q as the MMA's N) and the widened weights never pass through
// shared memory.
//
// Tiles.  The segments' lengths are on the device only, so every CTA builds
// the tile table itself from the offsets: expert e with c rows makes
// ceil(c / BMT) row tiles of equal height (rounded up to 16, the MMA's N
// step), each times ceil(N / 128) weight tiles, weight tiles fastest (the
// CTAs that run together share a row tile and sweep one expert's weights).
// A tile costs what its rows need: the MMA's N, the loaded boxes and the
// stored boxes follow its height.
//
// Persistent, one CTA per SM, warps by role (K in pieces of 64; a stage is H
// pieces, H = 2, or 4 for low tiles):
//   warp 0      weight producer: 256-deep K chunks of the FP4 tile (128-byte
//               rows, 128-byte swizzle) and their scales by TMA, WS-deep ring;
//   warp 1      TMEM allocator and MMA issuer (kind::f16, A from tensor memory);
//   warp 2      activation producer: a stage is one 3-D TMA box, rows x pieces,
//               of the smallest of three heights that covers the tile, RS-deep
//               ring;
//   4 H warps   transform: four warps widen piece h of every stage, lane l of
//               lane quarter q its weight row 32 q + l, in registers first and
//               then, once the MMAs of stage it - AS are done, into one of AS
//               tensor-memory slots;
//   8 warps     epilogue: a TMEM lane quarter each, every other 32-row box:
//               scale, bf16, and a TMA store of the 32 x 32 box through the
//               warp's own staging buffer.  A box that reaches past its
//               segment is stored row by row, so no row of another segment
//               or behind the last one is written.
//
// What bounds a stage, and what that led to (eight experts, 17664 rows x 7680
// x 1920, and, where weights dominate, 32 experts x 192 rows x 1920 x 7680;
// each figure as measured at its step, B200):
//   * the producers' issue: a TMA instruction costs its thread a hundred
//     cycles or two.  One lane picked by elect.sync issues (behind `lane == 0`
//     711 against 497 us at five per 64-deep stage), the weights come 256
//     deep, and weights and activations have a warp each: 388 us;
//   * the MMA thread: about 130 cycles for each barrier that it passes and
//     170 for its MMAs and commits, 450 a stage whatever the tile's height.
//     Ring positions instead of divisions, the abort flag only behind a
//     failed wait: 365 us; stages of two or four pieces with one commit for
//     activations and A slot, see the next;
//   * the slot's turn-around: MMA, commit, wait, widening, store.  Widening
//     before the wait leaves only the store in it: 343 us, and 144 us (165
//     before).
// Now: 349 to 359 us in different sessions (1450 to 1490 TFLOP/s, 0.85 to 0.87
// of the measured bf16 peak), the tensor pipe active 75% of the time on a case
// of 4416 rows.  Two sets of transform warps taking the stages in turn were
// slower (359 against 383 us): the issue slots are half used already.
// With few rows per expert the handshakes of a stage and the transform warps'
// instructions bound it (conversions, f16x2 products and byte permutes all run
// at 64 lanes a cycle and SM): 32 experts of 32 rows x 1920 x 7680 take 78 us
// against 41 for the weights' bytes, 61 us with neither loads nor conversions.
// All waits are bounded; on a timeout a role records it, drains its own
// copies or MMAs and leaves the loop, and the CTA frees its tensor memory.
#include "ql_common.cuh"
#include "gemm_common.cuh"
#include "launchers.h"
#include "segments.cuh"

namespace ql {

constexpr int kMaxExperts = 1024;

struct GroupedArgs {
  const int32_t* offsets;
  const int32_t* rows;       // scale of row r: row_scale[rows[r]]; null: row_scale[r]
  const float* row_scale;    // [rows_a]
  const float* g_w;          // [E]
  const uint8_t* sf;
  __nv_bfloat16* y;
  size_t expert_sf;
  int64_t rows_a, T;         // rows of row_scale, of Y
  int32_t E, N, K;
  int32_t tiles_n, num_kst, k_atoms;
  float alpha_mul;
  long long wait_limit;
  int* status;
};

template <int BMT, int RS, int WS, int H>
struct GroupedCfg {
  static constexpr int BK = 64 * H;                // K elements of a stage: H pieces of 64
  static constexpr int WK = 4 / H;                 // stages of a weight chunk (256 elements)
  static constexpr int NACC = 2;
  static constexpr int ACOLS = 32 * H;             // tensor-memory columns of an A slot
  static constexpr int FREE = (512 - NACC * BMT) / ACOLS;
  static constexpr int AS = FREE < RS ? FREE : RS; // A slots
  static constexpr int BOX1 = BMT == 192 ? 128 : BMT / 2;   // smaller activation boxes
  static constexpr int BOX2 = BMT == 192 ? 64 : BMT / 4;
  static constexpr int B_BYTES = H * BMT * 128;    // 64 f16 of K per row and piece
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int SF_BYTES = 4 * 512;
  static constexpr int OFF_B = 0;
  static constexpr int OFF_W = OFF_B + RS * B_BYTES;
  static constexpr int OFF_SF = OFF_W + WS * W_BYTES;
  static constexpr int OFF_C = OFF_SF + WS * SF_BYTES;
  static constexpr int OFF_TAB = OFF_C + 8 * 2 * kWarpBoxBytes;      // first tile and first row of each expert
  static constexpr int OFF_BAR = OFF_TAB + 2 * 4 * (kMaxExperts + 4);
  static constexpr int NBAR = 2 * RS + 2 * WS + AS + 2 * 2 + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static constexpr __host__ __device__ int box_rows(int n) { return n > BOX1 ? BMT : n > BOX2 ? BOX1 : BOX2; }
  static constexpr int EPI0 = 4 + 4 * H;           // first epilogue warp
  static constexpr int THREADS = (EPI0 + 8) * 32;
  static_assert(AS >= 2, "tensor memory budget");
  static_assert(H == 2 || H == 4, "a weight chunk is two stages or one");
  static_assert(BOX2 % 8 == 0, "whole swizzle atoms");
  static_assert(OFF_BAR % 8 == 0, "mbarrier alignment");
  static_assert(SMEM <= 232448, "shared memory budget");
};

// kind::f16: D = F32, A = B = F16, both K-major, M = 128, N = n (a multiple of 16)
__device__ __forceinline__ uint32_t grouped_idesc(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// Whether the phase with the given parity has completed (no suspension).
__device__ __forceinline__ bool mbar_test(uint32_t bar_addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar_addr), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

struct GroupedTile {
  int e, nb;       // expert, weight tile
  int row0, rows;  // rows [row0, row0 + rows) of Y
  int n;           // rows rounded up to the MMA's step
};

// Walks the tile table in ascending tile order.
struct TileCursor {
  const int* first;   // first row tile of each expert, [E] the total
  const int* lo;      // first row of each expert, [E] the end
  int e;
  __device__ __forceinline__ GroupedTile at(int t, int tiles_n, int bmt) {
    const int tt = t / tiles_n;
    while (first[e + 1] <= tt) ++e;
    const int count = lo[e + 1] - lo[e], nt = first[e + 1] - first[e];
    const int per = ((count + nt - 1) / nt + 15) & ~15;
    const int start = (tt - first[e]) * per;
    GroupedTile r;
    r.e = e;
    r.nb = t - tt * tiles_n;
    r.row0 = lo[e] + start;
    r.rows = min(per, count - start);
    r.n = (r.rows + 15) & ~15;
    return r;
  }
};

// Position in a ring of N slots: the slot and the phase parity of its use.
template <int N>
struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// Bounded wait of one thread; the abort flag is looked at only when the
// phase is not complete yet.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, long long limit, volatile int* abort_flag) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const long long t0 = clock64();
  while (*abort_flag == 0) {
    if (mbar_try_wait(a, parity)) return true;
    if (clock64() - t0 > limit) return false;
  }
  return false;
}

// The same for a warp: every lane looks, a few times; then one lane waits and
// all take its outcome.  (A suspended waiter wakes late: looking 64 times
// first took 17664 x 7680 x 1920 over eight experts from 365 to 349 us.  Not
// for the single-thread roles, whose looks cost the transform warps of their
// SM sub-partition issue slots: 377 us.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, long long limit, volatile int* abort_flag) {
  for (int i = 0; i < 64; ++i)
    if (__all_sync(0xffffffffu, mbar_test(smem_u32(bar), parity))) return true;
  int ok = 0;
  if (lane_id() == 0) ok = wait_or_abort(bar, parity, limit, abort_flag);
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

template <int BMT, int RS, int WS, int H>
__global__ void __launch_bounds__(GroupedCfg<BMT, RS, WS, H>::THREADS, 1)
    k_gemm_grouped(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_x1,
                   const __grid_constant__ CUtensorMap tm_x2, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_y, const GroupedArgs p) {
  using C = GroupedCfg<BMT, RS, WS, H>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1024(smem_raw);
  uint64_t* b_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* b_empty = b_full + RS;
  uint64_t* w_full = b_empty + RS;
  uint64_t* w_empty = w_full + WS;
  uint64_t* xf_full = w_empty + WS;
  uint64_t* tfull = xf_full + C::AS;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* s_first = reinterpret_cast<int*>(smem + C::OFF_TAB);
  int* s_lo = s_first + kMaxExperts + 4;

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();
  if (threadIdx.x == 0) {
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_x1);
    prefetch_tmap(&tm_x2);
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_y);
    for (int i = 0; i < RS; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
    for (int i = 0; i < WS; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_empty[i], 4 * H * C::WK);   // the transform warps x the chunk's stages
    }
    for (int i = 0; i < C::AS; ++i) mbar_init(&xf_full[i], 4 * H);   // the transform warps
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  pdl_wait();
  if (warp == 0) {   // the tile table
    int total = 0;
    int64_t carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + static_cast<int>(lane);
      int64_t lo, hi;
      warp_segments(p.offsets, p.E, p.T, e, carry, lo, hi);
      const int cnt = static_cast<int>(hi - lo), tiles = (cnt + BMT - 1) / BMT;
      const int end = warp_inclusive_sum(tiles);
      if (e < p.E) {
        s_first[e] = total + end - tiles;
        s_lo[e] = static_cast<int>(lo);
      }
      total += __shfl_sync(0xffffffffu, end, 31);
    }
    if (lane == 0) {
      s_first[p.E] = total;
      s_lo[p.E] = static_cast<int>(carry);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t a_slots = tmem + C::NACC * BMT;
  const int num_tiles = s_first[p.E] * p.tiles_n;
  TileCursor cur{s_first, s_lo, 0};
  const int chunks = (p.num_kst + C::WK - 1) / C::WK;

  if (warp == 0) {
    // ------------------------------------------------------------ weight producer
    if (elect_one()) {
      int it = 0;
      RingPos<WS> w;
      bool ok = true;
      for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
        const GroupedTile g = cur.at(t, p.tiles_n, BMT);
        const uint8_t* sf = p.sf + static_cast<size_t>(g.e) * p.expert_sf + static_cast<size_t>(g.nb) * p.k_atoms * 512;
        const int wrow = g.e * p.N + g.nb * 128;
        for (int c = 0; c < chunks; ++c, ++it, w.advance()) {
          if (!wait_or_abort(&w_empty[w.slot], w.phase ^ 1, p.wait_limit, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t sf_bytes = 512 * min(4, p.k_atoms - 4 * c);
          mbar_arrive_expect_tx(&w_full[w.slot], C::W_BYTES + sf_bytes);
          tma_load_2d(smem + C::OFF_W + w.slot * C::W_BYTES, &tm_w, &w_full[w.slot], c * 128, wrow);
          bulk_load(smem + C::OFF_SF + w.slot * C::SF_BYTES, sf + static_cast<size_t>(c) * C::SF_BYTES, sf_bytes,
                    &w_full[w.slot]);
        }
      }
      if (!ok) fail_timeout(p.status, abort_flag);
      drain_loads(w_full, it, WS, p.status);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ activation producer
    if (elect_one()) {
      int it = 0;
      RingPos<RS> b;
      bool ok = true;
      for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
        const GroupedTile g = cur.at(t, p.tiles_n, BMT);
        // the smallest box that covers the tile
        const CUtensorMap* tm = g.n > C::BOX1 ? &tm_x : g.n > C::BOX2 ? &tm_x1 : &tm_x2;
        const uint32_t bytes = 128 * H * C::box_rows(g.n);
        for (int ks = 0; ks < p.num_kst; ++ks, ++it, b.advance()) {
          if (!wait_or_abort(&b_empty[b.slot], b.phase ^ 1, p.wait_limit, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&b_full[b.slot], bytes);
          tma_load_3d(smem + C::OFF_B + b.slot * C::B_BYTES, tm, &b_full[b.slot], 0, g.row0, H * ks);
        }
      }
      if (!ok) fail_timeout(p.status, abort_flag);
      drain_loads(b_full, it, RS, p.status);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      RingPos<RS> b;
      RingPos<C::AS> a;
      RingPos<C::NACC> d;
      const uint64_t bdesc0 = smem_desc(smem_u32(smem + C::OFF_B), 0, 1024, kSwizzle128B);
      bool ok = true;
      for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x, d.advance()) {
        const int n = cur.at(t, p.tiles_n, BMT).n;
        const uint32_t idesc = grouped_idesc(n);
        const uint32_t piece = static_cast<uint32_t>(C::box_rows(n) * 128 >> 4);   // from one piece of a stage to the next
        if (!wait_or_abort(&tempty[d.slot], d.phase ^ 1, p.wait_limit, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem + d.slot * BMT;
        uint32_t accumulate = 0;
        for (int ks = 0; ks < p.num_kst; ++ks, b.advance(), a.advance()) {
          if (!wait_or_abort(&b_full[b.slot], b.phase, p.wait_limit, abort_flag) ||
              !wait_or_abort(&xf_full[a.slot], a.phase, p.wait_limit, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // the descriptor's address field counts 16-byte units and has room for all of shared memory
          const uint64_t bdesc = bdesc0 + static_cast<uint32_t>(b.slot * (C::B_BYTES >> 4));
          const uint32_t a_tmem = a_slots + C::ACOLS * a.slot;
          const int pieces = min(H, p.k_atoms - H * ks);
#pragma unroll
          for (int h = 0; h < H; ++h) {
            if (h < pieces) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                tc_mma_f16_ts(d_tmem, a_tmem + 32 * h + 8 * i, bdesc + h * piece + 2 * i, idesc, accumulate);
                accumulate = 1;
              }
            }
          }
          tc_commit(&b_empty[b.slot]);   // frees the activation stage and the A slot
        }
        if (!ok) break;
        tc_commit(&tfull[d.slot]);
      }
      if (!ok) fail_timeout(p.status, abort_flag);
      drain_mma(drain, p.status);
    }
  } else if (warp >= 4 && warp < C::EPI0) {
    // ------------------------------------------------------------ transform
    const uint32_t q = static_cast<uint32_t>(warp & 3);
    const uint32_t row = 32 * q + lane;
    const int piece = (warp - 4) >> 2;    // of the stage's K elements
    int it = 0;
    RingPos<C::AS> a;
    RingPos<RS> freed;                    // the stage whose MMAs free the slot: it - AS
    RingPos<WS> w;
    bool ok = true;
    for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
      for (int ks = 0; ks < p.num_kst; ++ks, ++it) {
        if (ks % C::WK == 0 && !warp_wait(&w_full[w.slot], w.phase, p.wait_limit, abort_flag)) {
          ok = false;
          break;
        }
        const int sub = H * (ks % C::WK) + piece;   // 64-element piece of the weight chunk (past K: zeros)
        // scale atom: byte (row % 32) * 16 + (row / 32) * 4 + k16 holds the block scale of K block k16
        const uint32_t sb4 = *reinterpret_cast<const uint32_t*>(smem + C::OFF_SF + w.slot * C::SF_BYTES + sub * 512 +
                                                                lane * 16 + q * 4);
        // 16-byte piece i of a swizzled 128-byte row sits at i ^ (row % 8)
        const uint8_t* wr = smem + C::OFF_W + w.slot * C::W_BYTES + row * 128;
        const uint4 c0 = *reinterpret_cast<const uint4*>(wr + (((2 * sub) ^ (row & 7)) << 4));
        const uint4 c1 = *reinterpret_cast<const uint4*>(wr + (((2 * sub + 1) ^ (row & 7)) << 4));
        const uint32_t cw[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        uint32_t v[32];
#pragma unroll
        for (int w8 = 0; w8 < 8; ++w8) {
          const __half2 s2 = e4m3x2_to_f16(w8 < 4 ? sb4 : sb4 >> 16);       // scales of words w8 & 4 .. + 3, two words each
          const __half2 s = (w8 & 2) ? __high2half2(s2) : __low2half2(s2);
          uint32_t h[4];
          fp4x8_to_f16(cw[w8], h);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[4 * w8 + j] = h2_bits(__hmul2(bits_h2(h[j]), s));
        }
        // the weights are widened in registers before the slot is waited for,
        // so a slot's turn-around is only the store
        if (it >= C::AS && !warp_wait(&b_empty[freed.slot], freed.phase, p.wait_limit, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        tmem_st32(a_slots + ((32 * q) << 16) + C::ACOLS * a.slot + 32 * piece, v);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        const bool last = ks % C::WK == C::WK - 1 || ks == p.num_kst - 1;   // of the chunk
        if (lane == 0) {
          mbar_arrive(&xf_full[a.slot]);
          // a chunk of one stage (the last one of some K) counts it twice
          mbar_arrive_n(&w_empty[w.slot], last && ks % C::WK == 0 ? C::WK : 1);
        }
        if (last) w.advance();
        if (it >= C::AS) freed.advance();
        a.advance();
        __syncwarp();   // the tcgen05 instructions need the whole warp together
      }
    }
    if (!ok && lane == 0) fail_timeout(p.status, abort_flag);
  } else if (warp >= C::EPI0) {
    // ------------------------------------------------------------ epilogue
    const uint32_t q = static_cast<uint32_t>(warp & 3);
    const int half = (warp - C::EPI0) >> 2;
    uint8_t* stage = smem + C::OFF_C + (warp - C::EPI0) * 2 * kWarpBoxBytes;
    int next = 0, local = 0;
    for (int t = blockIdx.x; t < num_tiles; t += gridDim.x, ++local) {
      const GroupedTile g = cur.at(t, p.tiles_n, BMT);
      const int acc = local % C::NACC;
      if (!warp_wait_uniform(&tfull[acc], (local / C::NACC) & 1, p.wait_limit, abort_flag, p.status)) break;
      tc_fence_after();
      const float alpha = __fmul_rn(ld_dep(p.g_w + g.e), p.alpha_mul);
      const int n0 = g.nb * 128 + 32 * static_cast<int>(q);
      const int boxes = n0 < p.N ? (g.rows + 31) >> 5 : 0;       // this warp's: half, half + 2, ...
      for (int c = half; c < boxes; c += 2) {
        const int m = 32 * c + static_cast<int>(lane);           // row of the tile
        float a_l = 0.f;
        if (m < g.rows) {
          int64_t src = static_cast<int64_t>(g.row0) + m;
          if (p.rows != nullptr) src = p.rows[src];
          if (src >= 0 && src < p.rows_a) a_l = __fmul_rn(alpha, ld_dep(p.row_scale + src));
        }
        uint32_t r[32];
        __syncwarp();   // the tcgen05 instructions need the whole warp together
        tmem_ld32(tmem + ((32 * q) << 16) + acc * BMT + 32 * c, r);
        tmem_ld_wait();
        if (c + 2 >= boxes) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
        }
        if (32 * c + 32 <= g.rows) {
          uint8_t* buf = stage + next * kWarpBoxBytes;
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(buf) + lane;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            dst[32 * j] = __float2bfloat16_rn(__fmul_rn(__shfl_sync(0xffffffffu, a_l, j), __uint_as_float(r[j])));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm_y, buf, n0, g.row0 + 32 * c);
            bulk_commit();
          }
          next ^= 1;
        } else {
          const int n = n0 + static_cast<int>(lane);
          __nv_bfloat16* dst = p.y + (static_cast<int64_t>(g.row0) + 32 * c) * p.N + n;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float v = __fmul_rn(__shfl_sync(0xffffffffu, a_l, j), __uint_as_float(r[j]));
            if (32 * c + j < g.rows && n < p.N) dst[static_cast<int64_t>(j) * p.N] = __float2bfloat16_rn(v);
          }
        }
      }
      if (half >= boxes) {   // no box: nothing was read
        tc_fence_before();
        if (lane == 0) mbar_arrive(&tempty[acc]);
      }
    }
    epilogue_warp_finish();
  }

  pdl_release();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int BMT, int RS, int WS, int H>
static ql_status launch_grouped_cfg(const void* a, const float* a_scales, int64_t rows_a, const int32_t* rows,
                                    const int32_t* offsets, int64_t T, const ql_experts* w, void* Y, cudaStream_t st,
                                    int* status) {
  using C = GroupedCfg<BMT, RS, WS, H>;
  const int N = w->N, K = w->K;
  const int64_t x_rows = rows != nullptr ? T : rows_a;
  // 64 values x rows x pieces of K: one box brings all pieces of a stage
  auto x_map = [&](CUtensorMap* map, uint32_t box_rows) {
    return make_tmap_3d(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a, 64, x_rows, K / 64, static_cast<int64_t>(K) * 2, 128, 64,
                        box_rows, H, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  CUtensorMap tx, tx1, tx2, tw, ty;
  if (!x_map(&tx, BMT) || !x_map(&tx1, C::BOX1) || !x_map(&tx2, C::BOX2) ||
      !make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w->codes, K / 2, static_cast<int64_t>(w->E) * N, K / 2,
                    128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, Y, N, T, static_cast<int64_t>(N) * 2, 32, 32,
                    CU_TENSOR_MAP_SWIZZLE_NONE))
    return QL_ERR_CUDA;
  GroupedArgs p{};
  GemmArgs limits{};
  fill_gemm_args(limits, T, N, K, 128, status);
  p.offsets = offsets;
  p.rows = rows;
  p.row_scale = a_scales;
  p.g_w = w->gscale;
  p.sf = static_cast<const uint8_t*>(w->sf);
  p.y = static_cast<__nv_bfloat16*>(Y);
  p.expert_sf = qlinear_sf_bytes(N, K);
  p.rows_a = rows_a;
  p.T = T;
  p.E = w->E;
  p.N = N;
  p.K = K;
  p.tiles_n = (N + 127) / 128;
  p.num_kst = (K + C::BK - 1) / C::BK;
  p.k_atoms = K / 64;
  p.alpha_mul = w->hadamard ? (1.0f / 128.0f) : 1.0f;
  p.wait_limit = limits.wait_limit;
  p.status = status;
  // the most tiles that the rows can make
  const int64_t tiles = most_row_tiles(T, w->E, BMT) * p.tiles_n;
  if (tiles > 0x7FFFFFFF - num_sms()) return QL_ERR_UNSUPPORTED_SHAPE;
  auto kern = k_gemm_grouped<BMT, RS, WS, H>;
  if (!set_smem_attr(reinterpret_cast<const void*>(kern), C::SMEM)) return QL_ERR_CUDA;
  const int grid = static_cast<int>(std::min<int64_t>(tiles, num_sms()));
  if (launch_pdl(kern, dim3(grid), dim3(C::THREADS), C::SMEM, st, 1, tx, tx1, tx2, tw, ty, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return QL_ERR_CUDA;
  }
  return QL_OK;
}

// ---------------------------------------------------------------------------
// Source rows into output order: out[r] = a[rows[r]] (zeros for a row that
// does not exist).  HBM: 2 bytes per value written, and read where a row is
// new to L2.  The product then loads whole boxes; gathering inside it was
// slower, since each row tile is loaded once per 128 columns of Y: 17664 x 7680 x 1920 took 974 us with four-row TMA
// gathers and 742 us with 16-byte asynchronous copies, against 388 us for
// rows in order.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreadsHbm) k_gather_rows(const uint4* a, const int32_t* rows, int64_t rows_a, int64_t T,
                                                             int32_t pieces, uint4* out) {
  pdl_wait();
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreadsHbm / 32);
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreadsHbm / 32) + (threadIdx.x >> 5); r < T; r += step) {
    const int32_t v = rows[r];
    const bool ok = v >= 0 && v < rows_a;
    const uint4* src = a + static_cast<int64_t>(ok ? v : 0) * pieces;
    uint4* dst = out + r * pieces;
#pragma unroll 4
    for (int32_t i = static_cast<int32_t>(lane_id()); i < pieces; i += 32)
      dst[i] = ok ? src[i] : make_uint4(0, 0, 0, 0);
  }
  pdl_release();
}

// Tile height by the rows per expert: a tall tile widens the weights once
// for more rows, a low one leaves room for longer K stages and a deeper
// weight ring.  64 experts 1408 x 2048 at 32 / 64 / 128 rows each on average:
// 64-row tiles 36 / 50 / 74 us, 128-row 43 / 46 / 59, 192-row 46 / 49 / 60;
// 32 experts 1920 x 7680: 78 / 97 / 164, 96 / 98 / 131, 110 / 113 / 129.
// Low tiles too where all of them run at once: a K step of theirs takes 0.63 us
// per 256 elements, one of the others 0.4 to 0.6 per 128.
static int grouped_tile_rows(int64_t T, int64_t E, int64_t N) {
  if (T <= 40 * E || most_row_tiles(T, E, 64) * ((N + 127) / 128) <= kEstimateSms) return 64;
  return T <= 100 * E ? 128 : 192;
}

// ns of the tiles beyond the launch, from the fullest SM's tiles.
int64_t grouped_tiles_ns(int64_t T, int64_t E, int64_t N, int64_t K) {
  const int rows = grouped_tile_rows(T, E, N);
  const int64_t sm_tiles = (most_row_tiles(T, E, rows) * ((N + 127) / 128) + kEstimateSms - 1) / kEstimateSms;
  return 2000 + sm_tiles * (rows == 64 ? (K + 255) / 256 * 630 : (K + 127) / 128 * 400);
}

ql_status launch_gemm_grouped(const void* a, const float* a_scales, int64_t rows_a, const int32_t* rows,
                              const int32_t* offsets, int64_t T, const ql_experts* w, void* Y, void* gathered,
                              cudaStream_t st, int* status) {
  const void* x = a;
  if (rows != nullptr) {
    const int64_t want = (T + kThreadsHbm / 32 - 1) / (kThreadsHbm / 32);   // a warp per row
    const int grid = static_cast<int>(std::min<int64_t>(want, 8ll * num_sms()));
    if (launch_pdl(k_gather_rows, dim3(grid), dim3(kThreadsHbm), 0, st, 1, static_cast<const uint4*>(a), rows, rows_a, T,
                   w->K / 8, static_cast<uint4*>(gathered)) != cudaSuccess) {
      (void)cudaGetLastError();
      return QL_ERR_CUDA;
    }
    x = gathered;
  }
  switch (grouped_tile_rows(T, w->E, w->N)) {
    case 64: return launch_grouped_cfg<64, 3, 4, 4>(x, a_scales, rows_a, rows, offsets, T, w, Y, st, status);
    case 128: return launch_grouped_cfg<128, 4, 3, 2>(x, a_scales, rows_a, rows, offsets, T, w, Y, st, status);
    default: return launch_grouped_cfg<192, 3, 2, 2>(x, a_scales, rows_a, rows, offsets, T, w, Y, st, status);
  }
}

}  // namespace ql
