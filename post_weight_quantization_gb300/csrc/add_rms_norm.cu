// The residual's addition and the RMS norm of a token's row, in one pass:
//
//   s = x + r,   r_out = s rounded to r's type,   y = s * rsqrt(mean(s^2) + eps) * w
//
// with the sum and the norm in fp32 (the norm is that of s before its rounding), and y in fp32, bf16,
// fp16 or in 8 bits: e4m3 with a scale per token, scale = max|y| / 448. There the norm's factor falls out of the
// codes, y / scale = s w * 448 / max|s w|, so that a code is one rounding (of s w) and its own.
//
// A row lies in the registers of its threads, eight consecutive values to a vector, V vectors a thread
// (vector i of thread t is t + i * threads), so X and R are read once and nothing is read twice. A row of at
// most 1024 values belongs to one warp, a longer one to a block; the sum of squares and the largest |s w|
// meet by shuffles and, in a block, by one trip through shared memory, in an order that the row's
// length alone decides.
//
// Bound: HBM, every value read once and written once. Measured, bf16 with residual: 16381 x 8192 into 8 bits 138 us (6.8 TB/s, a plain
// copy's rate), 4099 x 4096 24 us.
#include <algorithm>
#include <type_traits>

#include "elem.cuh"

namespace gptq {
namespace arn {

struct E4M3 { using T = uint8_t; };

// Two values to e4m3, the first in the low byte: to nearest even, at most 448, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}

// The larger one; a NaN, where one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

struct Params {
  const void* x;
  const void* r;               // NULL: no residual
  void* ro;
  const float* w;              // NULL: ones
  void* y;
  float* scale;
  long long ldx, ldr, ldro, ldy;
  long long T;
  int n8;                      // vectors of a row
  float eps, inv_d;
};

constexpr int ROWS = 4;                                    // rows of a block whose warps have a row each

template <typename EI>
struct Raw { uint4 v[std::is_same<EI, F32>::value ? 2 : 1]; };

template <typename EI>
__device__ __forceinline__ Raw<EI> load8(const void* base, long long at) {
  Raw<EI> r;
  const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const typename EI::T*>(base) + at);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r) / sizeof(uint4)); ++i) r.v[i] = p[i];
  return r;
}

// MOST: threads of a block at most, 0 where each warp has its own row
template <typename EI, typename EO, int V, int MOST>
__global__ void __launch_bounds__(MOST ? MOST : 32 * ROWS) add_rms_norm_kernel(Params p) {
  constexpr bool WARP = MOST == 0;
  using TI = typename EI::T;
  using TO = typename EO::T;
  constexpr bool BYTES = std::is_same<EO, E4M3>::value;
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long t = WARP ? (long long)blockIdx.x * ROWS + warp : (long long)blockIdx.x;
  if (t >= p.T) return;                                    // whole warps, and only where a warp has a row
  const int me = WARP ? lane : (int)threadIdx.x, step = WARP ? 32 : (int)blockDim.x;
  float s[V][8];
  // vectors in flight: all, but of fp32 in the longest rows, where 64 registers a thread do not hold them
  constexpr int AT = MOST == 1024 && std::is_same<EI, F32>::value ? 1 : V;
#pragma unroll
  for (int i0 = 0; i0 < V; i0 += AT) {
    Raw<EI> x[AT], r[AT];
#pragma unroll
    for (int j = 0; j < AT; ++j)
      if (me + (i0 + j) * step < p.n8) x[j] = load8<EI>(p.x, t * p.ldx + 8 * (me + (i0 + j) * step));
    if (p.r) {
#pragma unroll
      for (int j = 0; j < AT; ++j)
        if (me + (i0 + j) * step < p.n8) r[j] = load8<EI>(p.r, t * p.ldr + 8 * (me + (i0 + j) * step));
    }
#pragma unroll
    for (int j = 0; j < AT; ++j) {
      const int i = i0 + j;
      if (me + i * step < p.n8) {
        unpack8<EI>(&x[j], s[i]);
        if (p.r) {
          float u[8];
          unpack8<EI>(&r[j], u);
#pragma unroll
          for (int k = 0; k < 8; ++k) s[i][k] += u[k];
          pack8<EI>(reinterpret_cast<TI*>(p.ro) + t * p.ldro + 8 * (me + i * step), s[i]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) s[i][k] = 0.0f;
      }
    }
  }
  float ss = 0.0f, big = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(s[i][k], s[i][k], ss);
    if (BYTES) {
      if (p.w && me + i * step < p.n8) {
        float w[8];
        unpack8<F32>(p.w + 8 * (me + i * step), w);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[i][k] *= w[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) big = max_nan(big, fabsf(s[i][k]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (BYTES) big = max_nan(big, __shfl_xor_sync(0xffffffffu, big, o));
  }
  if (!WARP) {
    if (lane == 0) {
      red[0][warp] = ss;
      red[1][warp] = big;
    }
    __syncthreads();
    const bool in = lane < (int)(blockDim.x >> 5);
    ss = in ? red[0][lane] : 0.0f;
    big = in ? red[1][lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (BYTES) big = max_nan(big, __shfl_xor_sync(0xffffffffu, big, o));
    }
  }
  const float n = rsqrtf(fmaf(ss, p.inv_d, p.eps));
  TO* y = reinterpret_cast<TO*>(p.y) + t * p.ldy;
  if constexpr (BYTES) {
    // a row of zeros (or of values whose reciprocal fp32 does not hold) has codes and a scale of 0, whatever n is there;
    // a NaN, or an infinity times 0, is the row's maximum, and an infinity's n is 0, or its difference from itself (of a product
    // with a weight) no number: a scale and codes of NaN
    const float top = big < 0x1p-119f ? 0.0f : big, scale = top == 0.0f ? 0.0f : __fdiv_rn(top * n, 448.0f) + (top - top);
    // v * 448 / top, with the quotient's remainder put back (Markstein): correctly rounded, so a quotient halfway
    // between two codes stays there. A power of two keeps the steps in fp32's range.
    const float f = top > 0x1p64f ? 0x1p-64f : top < 0x1p-40f ? 0x1p64f : 1.0f, f448 = 448.0f * f, tf = top * f;
    const float inv = scale > 0.0f ? __fdiv_rn(1.0f, tf) : scale;
    if (me == 0) p.scale[t] = scale;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (me + i * step < p.n8) {
        uint32_t q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float c[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float a = s[i][2 * k + h] * f448, q0 = a * inv;
            c[h] = fmaf(fmaf(-q0, tf, a), inv, q0);
          }
          q[k] = e4m3x2(c[0], c[1]);
        }
        *reinterpret_cast<uint2*>(y + 8 * (me + i * step)) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (me + i * step < p.n8) {
        float w[8];
        if (p.w) unpack8<F32>(p.w + 8 * (me + i * step), w);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[i][k] = p.w ? s[i][k] * n * w[k] : s[i][k] * n;
        pack8<EO>(y + 8 * (me + i * step), s[i]);
      }
    }
  }
}

template <typename EI, typename EO, int V, int MOST>
void launch(const Params& p, cudaStream_t s) {
  const unsigned grid = (unsigned)(MOST ? p.T : (p.T + ROWS - 1) / ROWS);
  const int threads = MOST ? ((p.n8 + V - 1) / V + 31) / 32 * 32 : 32 * ROWS;
  add_rms_norm_kernel<EI, EO, V, MOST><<<grid, threads, 0, s>>>(p);
}

template <typename EI, typename EO>
void pick(const Params& p, cudaStream_t s) {
  const int n8 = p.n8;
  if (n8 <= 32) launch<EI, EO, 1, 0>(p, s);
  else if (n8 <= 64) launch<EI, EO, 2, 0>(p, s);
  else if (n8 <= 128) launch<EI, EO, 4, 0>(p, s);
  else if (n8 <= 512) launch<EI, EO, 2, 256>(p, s);
  else if (n8 <= 2048) launch<EI, EO, 4, 512>(p, s);
  else launch<EI, EO, 4, 1024>(p, s);
}

}  // namespace arn

gptq_status add_rms_norm_launch(const void* X, const void* R, int in_dtype, long long T, long long d, long long ldx,
                                long long ldr, const float* w, float eps, void* R_out, long long ldro, void* Y,
                                int out_dtype, long long ldy, float* y_scale, cudaStream_t s) {
  using namespace arn;
  Params p{};
  p.x = X; p.r = R; p.ro = R_out; p.w = w; p.y = Y; p.scale = y_scale;
  p.ldx = ldx; p.ldr = ldr; p.ldro = ldro; p.ldy = ldy;
  p.T = T; p.n8 = (int)(d / 8); p.eps = eps; p.inv_d = 1.0f / (float)d;
  with_dtype(in_dtype, [&](auto ei) {
    using EI = decltype(ei);
    if (out_dtype == GPTQ_E4M3) pick<EI, E4M3>(p, s);
    else with_dtype(out_dtype, [&](auto eo) { pick<EI, decltype(eo)>(p, s); });
  });
  count_launch();
  return check_launch("add_rms_norm_kernel");
}

}  // namespace gptq
