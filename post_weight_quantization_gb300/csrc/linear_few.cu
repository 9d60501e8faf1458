// A packed projection of a few tokens with what follows it (gptq_linear without adapters, groups of whole blocks of 128
// columns): Y[t][r] = act(x_scale[t] * sum_g scale[r][g] * sum_{j in g} X[t][j] (code[r][j] - zero[r][g]) + bias[r])
// * mul[t][r] + residual[t][r].
//
// A warp takes 16 or 32 rows and a run of the blocks, the CTA's others (and a cluster's) the other blocks. The products run on mma.sync
// m16n8k16 with the integers (code - zero) * 2^-6, exact in bf16, unpacked into the A fragments in registers: the codes
// go from HBM to registers and nowhere else. (On tcgen05 the integers have to pass through shared or tensor memory, by
// barriers whose waits cost about 0.45 us a block: 4096 x 4096, one token, 12.6 us, here 8.5.) A lane's 32 columns of a row are one
// load; MMA j takes its columns 4 j ... 4 j + 3, the same four for X, so that the order of k is a fixed permutation of
// the block's columns on both sides. A block's sums, times the row's scale, are added in fp32; the warps' and then the
// cluster's sums meet in shared memory in a fixed order.
//
// Bound: too little in flight. 28672 x 8192, one token: 41.0 us (3.2 TB/s), at 3.8 of 16 warps a scheduler, a third of whose time
// is spent on loads; issue slots 46 %, L1 58 % of its peak (a line a row for every 64 bytes of codes: a lane's fragment rows lie
// in eight lines), HBM 28 %. Copies through shared memory (cp.async) took twice as long.
#include <algorithm>
#include <type_traits>

#include "packed.cuh"

namespace gptq {
namespace lfw {

using namespace adp;

constexpr int WARPS = 8, N = 8, AHEAD = 2;               // warps of a CTA, tokens, blocks of a warp on their way

struct Params {
  const uint32_t* qweight;
  const float* scales;
  const float* zeros;
  const void* x;
  const float* x_scale;
  const float* bias;
  const void* mul;
  const void* residual;
  void* Y;
  long long ldx, ldy, ldm, ldr;
  int m, nb, T, G, gb, wpr, act, y_bf16, S;                // nb: blocks of a row, gb: of a group; S: CTAs that share rows
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 values to two bf16 pairs, exactly.
__device__ __forceinline__ void widen4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  uint32_t h[2];
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[0]) : "h"((uint16_t)v));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[1]) : "h"((uint16_t)(v >> 16)));
  uint32_t* to[2] = {&lo, &hi};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    *to[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
}

// RT: tiles of 16 rows of a warp, which share X's fragments
template <int BITS, int RT, bool BYTES>
__global__ void __launch_bounds__(WARPS * 32, 2) linear_few_kernel(Params p) {
  constexpr int ROWS = 16 * RT, PAD = N + 1;
  __shared__ float red[WARPS][ROWS * PAD];
  __shared__ float part[ROWS * PAD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = p.S > 1 ? (int)cluster_ctarank() : 0, r0 = (int)(blockIdx.x / p.S) * ROWS;
  const int c0 = (int)((long long)p.nb * rank / p.S), c1 = (int)((long long)p.nb * (rank + 1) / p.S);
  const int b0 = c0 + (c1 - c0) * warp / WARPS, b1 = c0 + (c1 - c0) * (warp + 1) / WARPS;
  const uint32_t* wp[RT][2];
  const float *sp[RT][2], *zp[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {                          // rows past the end repeat the last one
      const long long row = min(r0 + 16 * i + 8 * h + g, p.m - 1);
      wp[i][h] = p.qweight + row * p.wpr + t * BITS;
      sp[i][h] = p.scales + row * p.G;
      zp[i][h] = p.zeros + row * p.G;
    }
  using TX = typename std::conditional<BYTES, uint8_t, uint16_t>::type;
  const TX* xp = reinterpret_cast<const TX*>(p.x) + (long long)min(g, p.T - 1) * p.ldx + 32 * t;    // tokens past the end too

  float run[RT][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) run[i][k] = 0.0f;

  // the next blocks' codes are on their way while one is multiplied
  uint32_t w[AHEAD][RT][2][BITS];
  auto load = [&](int b, int to, int i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) load_words<BITS>(wp[i][h] + (long long)b * (4 * BITS), w[to][i][h]);
  };
  // A row's scale and zero of four blocks in its four lanes, the next four's on their way: a load for each block and row
  // would ask L1 for as many lines as the codes do
  float sc[RT][2], ze[RT][2], sc_next[RT][2], ze_next[RT][2];
  auto load_groups = [&](int b) {
    const int grp = (p.gb == 1 ? (b & ~3) + t : ((b & ~3) + t) / p.gb), at = min(grp, p.G - 1);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sc_next[i][h] = __ldg(sp[i][h] + at);
        ze_next[i][h] = __ldg(zp[i][h] + at);
      }
  };
  load_groups(b0);
#pragma unroll
  for (int a = 0; a < AHEAD; ++a)
#pragma unroll
    for (int i = 0; i < RT; ++i)
      if (b0 + a < b1) load(b0 + a, a, i);
  for (int b = b0; b < b1; b += AHEAD) {
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      if (b + a >= b1) break;
      if (((b + a) & 3) == 0 || b + a == b0) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            sc[i][h] = sc_next[i][h];
            ze[i][h] = ze_next[i][h];
          }
        load_groups(b + a + 4);
      }
      uint32_t x[16];                                      // 32 columns of the lane's token, pairs
      const TX* at = xp + (long long)(b + a) * KB;
      if constexpr (BYTES) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(at) + k);
          widen4(v.x, x[8 * k], x[8 * k + 1]);
          widen4(v.y, x[8 * k + 2], x[8 * k + 3]);
          widen4(v.z, x[8 * k + 4], x[8 * k + 5]);
          widen4(v.w, x[8 * k + 6], x[8 * k + 7]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(at) + k);
          x[4 * k] = v.x; x[4 * k + 1] = v.y; x[4 * k + 2] = v.z; x[4 * k + 3] = v.w;
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        uint32_t o[2][16];
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int from = (lane & ~3) | ((b + a) & 3);
          unpack32<BITS>(w[a][i][h], neg_zero(__shfl_sync(0xffffffffu, ze[i][h], from)), o[h]);
          f[h] = 64.0f * __shfl_sync(0xffffffffu, sc[i][h], from);
        }
        if (b + a + AHEAD < b1) load(b + a + AHEAD, a, i);
        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 8; ++j) mma(c, o[0][2 * j], o[1][2 * j], o[0][2 * j + 1], o[1][2 * j + 1], x[2 * j], x[2 * j + 1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) run[i][k] = fmaf(c[k], f[k >> 1], run[i][k]);
      }
    }
  }
  // ---- the warps' sums, then the cluster's
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) red[warp][(16 * i + 8 * (k >> 1) + g) * PAD + 2 * t + (k & 1)] = run[i][k];
  __syncthreads();
  const int total = ROWS * min(N, p.T);                    // outputs: rows fastest
  for (int o = threadIdx.x; o < total; o += WARPS * 32) {
    const int at = (o % ROWS) * PAD + o / ROWS;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) v += red[k][at];
    part[at] = v;
  }
  if (p.S > 1) {
    __syncwarp();                                          // the loop's passes differ within a warp
    cluster_sync();
  } else {
    __syncthreads();
  }
  for (int o = rank * WARPS * 32 + (int)threadIdx.x; o < total; o += p.S * WARPS * 32) {
    const int r = o % ROWS, tok = o / ROWS, row = r0 + r;
    if (row >= p.m) continue;
    const float mul = p.mul ? read_y(p.mul, tok * p.ldm + row, p.y_bf16) : 1.0f;
    const float res = p.residual ? read_y(p.residual, tok * p.ldr + row, p.y_bf16) : 0.0f;
    float v = 0.0f;
    if (p.S == 1) {
      v = part[r * PAD + tok];
    } else {
      const uint32_t at = smem_u32(&part[r * PAD + tok]);
      for (int k = 0; k < p.S; ++k) {
        float y;
        asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                     : "=f"(y)
                     : "r"(at), "r"(k));
        v += y;
      }
    }
    v = activate(fmaf(v, p.x_scale ? p.x_scale[tok] : 1.0f, p.bias ? p.bias[row] : 0.0f), p.act);
    if (p.mul) v *= mul;
    if (p.residual) v += res;
    if (p.y_bf16) reinterpret_cast<__nv_bfloat16*>(p.Y)[tok * p.ldy + row] = __float2bfloat16_rn(v);
    else reinterpret_cast<float*>(p.Y)[tok * p.ldy + row] = v;
  }
  if (p.S > 1) {
    __syncwarp();
    cluster_sync();                                        // nobody leaves while its sums are read
  }
}

template <int BITS, int RT, bool BYTES>
gptq_status launch(Params p, cudaStream_t s) {
  const long long tiles = (p.m + 16 * RT - 1) / (16 * RT);
  p.S = 1;
  while (p.S < 8 && 2 * p.S * tiles <= 2LL * sm_count() && 2 * p.S * WARPS <= p.nb) p.S *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * p.S));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, linear_few_kernel<BITS, RT, BYTES>, p);
  count_launch();
  return check_launch("linear_few_kernel");
}

// 32 rows a warp where there is work enough for all SMs: X's fragments serve twice. Measured at 4 bits, one token, in us,
// 16 / 32 rows: 28672 x 8192 47.4 / 41.0, 8192 x 28672 47.4 / 43.4, 11008 x 4096 16.7 / 18.0, 4096 x 4096 8.5 / 10.5.
template <int BITS, bool BYTES>
gptq_status pick(const Params& p, cudaStream_t s) {
  return (long long)p.m * p.nb > (1 << 19) ? launch<BITS, 2, BYTES>(p, s) : launch<BITS, 1, BYTES>(p, s);
}
template <bool BYTES>
gptq_status pick(int bits, const Params& p, cudaStream_t s) {
  switch (bits) {
    case 2: return pick<2, BYTES>(p, s);
    case 3: return pick<3, BYTES>(p, s);
    case 4: return pick<4, BYTES>(p, s);
    default: return pick<8, BYTES>(p, s);
  }
}

}  // namespace lfw

// Up to 8 tokens in bf16, or in e4m3 (`bytes`); group_size -1 or a multiple of 128, d a multiple of 128. The arguments
// are checked.
gptq_status linear_few_launch(const uint32_t* qweight, const float* scales, const float* zeros, long long m, long long d,
                              int bits, int group_size, const void* X, bool bytes, long long T, long long ldx,
                              const float* x_scale, const float* bias, int act, const void* mul, long long ldm,
                              const void* residual, long long ldr, void* Y, int y_dtype, long long ldy, cudaStream_t s) {
  using namespace lfw;
  Params p{};
  p.qweight = qweight; p.scales = scales; p.zeros = zeros; p.x = X; p.x_scale = x_scale; p.bias = bias; p.mul = mul;
  p.residual = residual; p.Y = Y; p.ldx = ldx; p.ldy = ldy; p.ldm = ldm; p.ldr = ldr;
  const long long gs = group_size < 0 ? d : group_size;
  p.m = (int)m; p.nb = (int)(d / KB); p.T = (int)T; p.G = (int)(d / gs); p.gb = (int)(gs / KB);
  p.wpr = (int)(d / 32 * bits);
  p.act = act; p.y_bf16 = y_dtype == GPTQ_BF16;
  return bytes ? pick<true>(bits, p, s) : pick<false>(bits, p, s);
}

}  // namespace gptq
