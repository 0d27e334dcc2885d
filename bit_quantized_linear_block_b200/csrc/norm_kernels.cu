// Residual addition, RMS norm and per-token quantization of the result, in
// one pass over the row: what stands before a quantized linear layer in a
// decoder block.
//
//   h = bf16(x + r)                      (x when there is no residual)
//   rstd = RN32(1 / sqrt(sum h^2 / K + eps))
//   y = bf16(RN(RN(h rstd) gamma))
//   z = H_128 y per 128-element block    (y when hadamard is 0)
//   s = RN(max|z| / qmax), q = rint(RN(z RN(qmax / max|z|)))
//
// The roundings of h and y to bf16 are the block's activation type, so the
// codes are bit for bit those of the per-token quantizer on y.  The sum of
// squares is held in fp64: every h^2 is exact there and the order of the
// additions moves the sum by about 2^-52, so rstd does not depend on how the
// row is split over threads (an fp32 sum would move the last bit of rstd and
// with it codes next to a rounding border).
//
// Bound: HBM (7 to 10 bytes per element) for bf16 output: 32760 x 5120 with a
// residual 194.5 us, 6.9 TB/s.  The codes add the rotation, the maximum and the
// rounding, and issue slots bound them (72% active): 17776 x 1920 to int8 47.3
// us with a residual and the norm's output left out, 5.0 TB/s.  A row belongs to W warps; a thread
// holds V vectors of 16 elements from the load to the codes, so the row is
// read once and written once, and the only exchanges are two reductions over
// the row.  In a 128-element Hadamard block (8 neighbouring threads) thread
// u holds the 8-element chunks u and u + 8: both loads and all stores of a
// warp cover whole 128-byte lines, distances 1, 2, 4 are packed f32x2
// butterflies over the two chunks, 8, 16, 32 are lane exchanges and 64 is
// inside a pair.
#include <type_traits>

#include "ql_common.cuh"
#include "gemm_common.cuh"
#include "launchers.h"

namespace ql {

namespace {

constexpr int kNormMaxThreads = 512;
constexpr int kNormThreads3 = 256;   // with three vectors per thread: 85 registers, three CTAs on an SM

struct NormArgs {
  const uint8_t* x;
  const uint8_t* residual;      // null: no residual
  const uint8_t* gamma;
  uint8_t* residual_out;        // h, or null
  uint8_t* norm_out;            // y, or null
  uint8_t* codes;
  float* scales;
  int64_t M;
  int32_t K, hadamard, qmax;
  int32_t warps_per_row, rows_per_cta;
  double eps, k_inv;            // k_inv = 1 / K
};

enum NormOut { kOutInt8 = 0, kOutF16 = 1, kOutBf16 = 2 };

// Sylvester butterflies in the order 1, 2, 4, ..., 64, each rounded to fp32,
// on P[j] = (z_{8u + j}, z_{64 + 8u + j}), u = lane % 8.
__device__ __forceinline__ void fwht128_chunks(float2 (&P)[8]) {
  const float2 m1 = make_float2(-1.f, -1.f);
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if ((j & s) == 0) {
        const float2 a = P[j], b = P[j + s];
        P[j] = __fadd2_rn(a, b);
        P[j + s] = __ffma2_rn(b, m1, a);   // a - b: one rounding of the exact difference
      }
    }
  }
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) {
    const float sg = (lane_id() & s) ? -1.f : 1.f;
    const float2 sg2 = make_float2(sg, sg);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float2 o;
      o.x = __shfl_xor_sync(0xffffffffu, P[j].x, s);
      o.y = __shfl_xor_sync(0xffffffffu, P[j].y, s);
      P[j] = __ffma2_rn(P[j], sg2, o);     // lower lane: own + other, upper lane: other - own
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = P[j].x, b = P[j].y;
    P[j] = make_float2(__fadd_rn(a, b), __fsub_rn(a, b));
  }
}

// 1 / sqrt(v) rounded to fp32.  An fp32 estimate (about 2^-22) and two Newton
// steps r <- r (3/2 - v r^2 / 2) in fp64 leave about 2^-52; v beyond fp32's
// comfortable range takes the fp64 functions.
__device__ __forceinline__ float rsqrt_f64(double v) {
  if (v > 1e-30 && v < 1e30) {
    double r = static_cast<double>(rsqrtf(static_cast<float>(v)));
    const double hv = 0.5 * v;
    r = r * fma(-hv * r, r, 1.5);
    r = r * fma(-hv * r, r, 1.5);
    return static_cast<float>(r);
  }
  return static_cast<float>(1.0 / sqrt(v));
}

// Two bf16 sums, each the exact sum rounded once.  (Rounding it to fp32
// first gives the same: a sum of two 8-bit significands that lies near a
// bf16 border has at most 17 bits and is exact in fp32.)
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 s = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&s);
}

// RN(x inv) + 1.5 2^23, whose low mantissa bits are rint(RN(x inv)) for a
// product below 2^22 (here at most qmax + 1/2): full-rate adds where the
// float-to-int conversion runs at an eighth of it.  The product is rounded by
// itself: a packed multiply and two single adds cannot be contracted.  (Packed
// multiplies here and in the norm: 17776 x 1920 to int8 39.8 against 42.5 us.)
constexpr float kRoundMagic = 12582912.0f;
__device__ __forceinline__ float2 round_magic(float2 x, float inv) {
  const float2 p = __fmul2_rn(x, make_float2(inv, inv));
  return make_float2(__fadd_rn(p.x, kRoundMagic), __fadd_rn(p.y, kRoundMagic));
}

// Barrier of one row's warps.
__device__ __forceinline__ void row_sync(int row_slot, int warps) {
  if (warps == 1) __syncwarp();
  else named_bar_sync(1 + row_slot, 32 * warps);
}

}  // namespace

// L lanes of a warp hold a row (32: whole warps, one or more).
template <int V, int OUT, int L>
__global__ void __launch_bounds__(V == 3 ? kNormThreads3 : kNormMaxThreads, V <= 2 ? 2 : V == 3 ? 3 : 1) k_norm_quantize(const NormArgs p) {
  __shared__ double s_sum[kNormMaxThreads / 32];
  __shared__ float s_max[kNormMaxThreads / 32];
  const int warps = p.warps_per_row;             // blockDim.x / 32
  const uint32_t lane = lane_id();
  const int slot = threadIdx.y * (32 / L) + (L < 32 ? static_cast<int>(lane) / L : 0);   // row of this CTA
  const int t = L < 32 ? static_cast<int>(lane) % L : threadIdx.x;                       // thread within the row
  const int warp = threadIdx.y * warps + (threadIdx.x >> 5);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * p.rows_per_cta + slot;
  pdl_wait();
  const bool live = row < p.M;                   // uniform over a row's warps
  if (L < 32 ? __any_sync(0xffffffffu, live) : live) {
    const int64_t base = row * p.K;              // element offset of the row
    const int nvec = p.K >> 4;                   // 16-element vectors, a multiple of 8
    // element offset of this thread's first chunk of vector v; the second is 64 further
    auto offset = [&](int v) { return 128 * ((t + v * 32 * warps) >> 3) + 8 * (t & 7); };
    auto active = [&](int v) { return (L == 32 || live) && t + v * 32 * warps < nvec; };
    uint4 h[V][2];
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v][0] = h[v][1] = make_uint4(0, 0, 0, 0);
      if (active(v)) {
        const int64_t o = 2 * (base + offset(v));
        h[v][0] = *reinterpret_cast<const uint4*>(p.x + o);
        h[v][1] = *reinterpret_cast<const uint4*>(p.x + o + 128);
      }
    }
    if (p.residual != nullptr) {
      uint4 r[V][2];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        r[v][0] = r[v][1] = make_uint4(0, 0, 0, 0);
        if (active(v)) {
          const int64_t o = 2 * (base + offset(v));
          r[v][0] = *reinterpret_cast<const uint4*>(p.residual + o);
          r[v][1] = *reinterpret_cast<const uint4*>(p.residual + o + 128);
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t* hw = reinterpret_cast<uint32_t*>(&h[v][c]);
          const uint32_t* rw = reinterpret_cast<const uint32_t*>(&r[v][c]);
#pragma unroll
          for (int i = 0; i < 4; ++i) hw[i] = add_bf16x2(hw[i], rw[i]);
          if (p.residual_out != nullptr && active(v))
            *reinterpret_cast<uint4*>(p.residual_out + 2 * (base + offset(v)) + 128 * c) = h[v][c];
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t* hw = reinterpret_cast<const uint32_t*>(&h[v][c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double a = bf16_lo(hw[i]), b = bf16_hi(hw[i]);
          sum = fma(a, a, sum);
          sum = fma(b, b, sum);
        }
      }
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (L == 32 && warps > 1) {
      if (lane == 0) s_sum[warp] = sum;
      row_sync(slot, warps);
      sum = 0.0;
      for (int w = 0; w < warps; ++w) sum += s_sum[slot * warps + w];
    }
    const float rstd = rsqrt_f64(sum * p.k_inv + p.eps);

    float2 P[V][8];
    float m = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint4 y[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint4 g = make_uint4(0, 0, 0, 0);
        if (active(v)) g = *reinterpret_cast<const uint4*>(p.gamma + 2 * offset(v) + 128 * c);
        const uint32_t* hw = reinterpret_cast<const uint32_t*>(&h[v][c]);
        const uint32_t* gw = reinterpret_cast<const uint32_t*>(&g);
        uint32_t* yw = reinterpret_cast<uint32_t*>(&y[c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 n = __fmul2_rn(__fmul2_rn(make_float2(bf16_lo(hw[i]), bf16_hi(hw[i])), make_float2(rstd, rstd)),
                                      make_float2(bf16_lo(gw[i]), bf16_hi(gw[i])));
          yw[i] = pack_bf16x2(n.x, n.y);
        }
      }
      if (active(v)) {
        const int64_t o = 2 * (base + offset(v));
        uint8_t* dst = OUT == kOutBf16 ? p.codes : p.norm_out;
        if (dst != nullptr) {
          *reinterpret_cast<uint4*>(dst + o) = y[0];
          *reinterpret_cast<uint4*>(dst + o + 128) = y[1];
        }
      }
      if constexpr (OUT != kOutBf16) {
        const uint32_t* y0 = reinterpret_cast<const uint32_t*>(&y[0]);
        const uint32_t* y1 = reinterpret_cast<const uint32_t*>(&y[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          P[v][2 * i] = make_float2(bf16_lo(y0[i]), bf16_lo(y1[i]));
          P[v][2 * i + 1] = make_float2(bf16_hi(y0[i]), bf16_hi(y1[i]));
        }
        if (p.hadamard) fwht128_chunks(P[v]);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmax3(m, fabsf(P[v][j].x), fabsf(P[v][j].y));
      }
    }
    if constexpr (OUT != kOutBf16) {
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (L == 32 && warps > 1) {
        if (lane == 0) s_max[warp] = m;
        row_sync(slot, warps);
        m = 0.f;
        for (int w = 0; w < warps; ++w) m = fmaxf(m, s_max[slot * warps + w]);
      }
      const float fq = static_cast<float>(p.qmax);
      // a maximum so small that qmax over it is no fp32 number: the step 2^-128,
      // a product with FLT_MAX and finite codes
      const float inv = (m == 0.f) ? 0.f : fminf(__fdiv_rn(fq, m), 3.402823466e38f);
      if (t == 0 && (L == 32 || live)) p.scales[row] = (m == 0.f) ? 0.f : fmaxf(__fdiv_rn(m, fq), 2.938735877e-39f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!active(v)) continue;
        const int64_t o = base + offset(v);
        float2 q[8];   // rounded codes plus the magic constant
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = round_magic(P[v][j], inv);
        if constexpr (OUT == kOutF16) {
          // the code itself (zero as +0), two per f16x2 convert (integers up to 127: exact)
          uint4 c[2];
          uint32_t* c0 = reinterpret_cast<uint32_t*>(&c[0]);
          uint32_t* c1 = reinterpret_cast<uint32_t*>(&c[1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            c0[i] = h2_bits(__floats2half2_rn(__fsub_rn(q[2 * i].x, kRoundMagic), __fsub_rn(q[2 * i + 1].x, kRoundMagic)));
            c1[i] = h2_bits(__floats2half2_rn(__fsub_rn(q[2 * i].y, kRoundMagic), __fsub_rn(q[2 * i + 1].y, kRoundMagic)));
          }
          *reinterpret_cast<uint4*>(p.codes + 2 * o) = c[0];
          *reinterpret_cast<uint4*>(p.codes + 2 * o + 128) = c[1];
        } else {
          auto pack4 = [](float a0, float a1, float a2, float a3) {
            const uint32_t lo = __byte_perm(__float_as_uint(a0), __float_as_uint(a1), 0x0040);   // the low bytes
            const uint32_t hi = __byte_perm(__float_as_uint(a2), __float_as_uint(a3), 0x0040);
            return __byte_perm(lo, hi, 0x5410);
          };
          *reinterpret_cast<uint2*>(p.codes + o) =
              make_uint2(pack4(q[0].x, q[1].x, q[2].x, q[3].x), pack4(q[4].x, q[5].x, q[6].x, q[7].x));
          *reinterpret_cast<uint2*>(p.codes + o + 64) =
              make_uint2(pack4(q[0].y, q[1].y, q[2].y, q[3].y), pack4(q[4].y, q[5].y, q[6].y, q[7].y));
        }
      }
    }
  }
  pdl_release();
}

ql_status launch_norm_quantize(const void* x, const void* residual, const void* gamma, int64_t M, int32_t K, float eps,
                               int out_kind, int hadamard, int qmax, void* residual_out, void* norm_out, void* codes,
                               float* scales, cudaStream_t st) {
  if (M == 0) return QL_OK;
  if (K > 4 * 16 * kNormMaxThreads) return QL_ERR_UNSUPPORTED_SHAPE;
  // Vectors per thread V, and with them the warps of a row.  Few rows: the
  // smallest V whose warps still run together, about 20 on an SM (148 x 4096
  // to int8, with a residual as all of these: 2.9 us at V = 1, 3.9 at 2, 4.5 at
  // 3; 600 x 2304 5.3, 5.1, 5.8).  Many rows: a warp costs about as much for
  // its part of the row's reductions, root and divisions as for a third of a
  // vector, and idle lanes cost what busy ones do, so the least of
  // warps (1 + 3 V): 17776 x 1024 30, 25, 32 us at V = 1, 2, 3, x 1536 49, 44,
  // 36, x 1920 55, 47, 62, x 2560 91, 72, 66 (one vector is behind wherever a row
  // needs two warps).  Four vectors have half the warps on an SM and only take
  // rows that need them.
  auto warps_for = [&](int V) { return (K / 16 + 32 * V - 1) / (32 * V); };
  auto fits = [&](int V) { return warps_for(V) <= (V == 3 ? kNormThreads3 : kNormMaxThreads) / 32; };
  int V = 4, least = INT32_MAX;
  for (int v = 1; v <= 3; ++v) {
    if (!fits(v)) continue;
    if (v <= 2 && M * warps_for(v) <= 20ll * num_sms()) {
      V = v;
      break;
    }
    const int cost = warps_for(v) * (1 + 3 * v);
    if (v == 1 && cost > 4) continue;
    if (cost < least) {
      least = cost;
      V = v;
    }
  }
  NormArgs p{};
  p.x = static_cast<const uint8_t*>(x);
  p.residual = static_cast<const uint8_t*>(residual);
  p.gamma = static_cast<const uint8_t*>(gamma);
  p.residual_out = static_cast<uint8_t*>(residual_out);
  p.norm_out = static_cast<uint8_t*>(norm_out);
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = scales;
  p.M = M;
  p.K = K;
  p.hadamard = hadamard;
  p.qmax = qmax;
  p.eps = static_cast<double>(eps);
  p.k_inv = 1.0 / static_cast<double>(K);
  p.warps_per_row = warps_for(V);
  const int L = K <= 128 ? 8 : K <= 256 ? 16 : 32;     // rows of 128 and 256 share a warp: 65536 x 128 to int8 10.5 us against 37.8
  const int slots = std::max(1, 8 / p.warps_per_row);  // short rows share a CTA of up to 8 warps
  p.rows_per_cta = slots * (32 / L);
  const int64_t grid = (M + p.rows_per_cta - 1) / p.rows_per_cta;
  auto pick = [&](auto out) -> void (*)(NormArgs) {
    constexpr int OUT = decltype(out)::value;
    if (L == 8) return k_norm_quantize<1, OUT, 8>;
    if (L == 16) return k_norm_quantize<1, OUT, 16>;
    return V == 1 ? k_norm_quantize<1, OUT, 32> : V == 2 ? k_norm_quantize<2, OUT, 32> : V == 3 ? k_norm_quantize<3, OUT, 32> : k_norm_quantize<4, OUT, 32>;
  };
  using std::integral_constant;
  void (*kern)(NormArgs) = out_kind == kOutInt8  ? pick(integral_constant<int, kOutInt8>{})
                           : out_kind == kOutF16 ? pick(integral_constant<int, kOutF16>{})
                                                 : pick(integral_constant<int, kOutBf16>{});
  if (launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(32 * p.warps_per_row, slots), 0, st, 1, p) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return QL_ERR_CUDA;
  }
  return QL_OK;
}

}  // namespace ql
