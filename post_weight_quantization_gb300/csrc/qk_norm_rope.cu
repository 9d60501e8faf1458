// The RMS norm of every query and key head and the position rotation, in one pass.
//
//   n = x * rsqrt(mean(x^2) + eps) * w,   then every pair (n_i, n_j) turned by the angle of
//   its position: (n_i c - n_j s, n_j c + n_i s)
//
// A row (one head of one token) lies in D / 8 of LPR lanes. A lane holds two runs of four
// values: for half-split pairs the same four places of the two halves of the rotated part
// (or of the part that is not rotated), for interleaved pairs eight in a row. Both members
// of every pair are in one lane, so a rotation needs no shuffle and four angles; the mean is
// log2(LPR) shuffles. Arithmetic is fp32; the one rounding is the store.
//
// Bound: HBM bandwidth (every value read once and written once). A warp takes one token and a
// strided set of its head blocks, NB rows per lane group each: the token's angles and the
// weights are read once for all of them, and a block's loads are in flight while the block
// before is computed. Measured, 16381 tokens of 64 + 8 heads of 128, bf16: 106 us, 5.75 TB/s, 85 % of
// a plain copy's rate.
#include <algorithm>
#include <type_traits>

#include "elem.cuh"

namespace gptq {
namespace qkr {

constexpr int WARPS = 4, NB = 4;

struct Params {
  const void* x[2];            // Q, K
  void* y[2];
  const float* w[2];
  long long ldx[2], ldy[2];
  int heads[2];
  int blocks[2];               // head blocks per token
  uint32_t T, parts;           // tokens, warps per token
  int D, rot;
  float eps;
  const float* cosv;
  const float* sinv;
  const int* pos;
  long long n_pos;
};

template <typename EI, typename EO, int LPR, bool INTERLEAVED>
__global__ void __launch_bounds__(WARPS * 32, std::is_same<EI, F32>::value ? 5 : 8) qk_norm_rope_kernel(Params p, int* __restrict__ err) {
  using TI = typename EI::T;
  using TO = typename EO::T;
  constexpr int RPW = 32 / LPR;                       // rows per warp at once
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const uint32_t unit = blockIdx.x * WARPS + (threadIdx.x >> 5), t = unit / p.parts;
  if (t >= p.T) return;
  const bool in = 8 * l < p.D;
  // the lane's two runs of four values
  int ca, cb;
  const int lr = l - p.rot / 8;
  if (INTERLEAVED) { ca = 8 * l; cb = ca + 4; }
  else if (lr < 0) { ca = 4 * l; cb = ca + p.rot / 2; }
  else { ca = p.rot + 4 * lr; cb = ca + (p.D - p.rot) / 2; }
  const bool turns = lr < 0;
  float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sn[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (p.rot) {
    const int pos = p.pos[t];
    if (pos < 0 || pos >= p.n_pos) {
      if (lane == 0) report_device_error(err, DEVERR_INDEX);
    } else if (turns) {
      unpack4<F32>(p.cosv + (long long)pos * (p.rot / 2) + 4 * l, cs);
      unpack4<F32>(p.sinv + (long long)pos * (p.rot / 2) + 4 * l, sn);
    }
  }
  const float inv_d = 1.0f / (float)p.D;
  const int nb = p.blocks[0] + p.blocks[1];
  int hb = (int)(unit - t * p.parts);

  // rows of block b in this lane: heads (b - first block of its tensor) * RPW * NB + sub + RPW i
  using RT = typename Raw4<EI>::T;
  RT raw[NB][2];
  auto load = [&](int b) {
    const int s = b >= p.blocks[0] ? 1 : 0, h0 = (b - (s ? p.blocks[0] : 0)) * (RPW * NB) + sub;
    const TI* x = reinterpret_cast<const TI*>(s ? p.x[1] : p.x[0]) + t * (s ? p.ldx[1] : p.ldx[0]);
    const int heads = s ? p.heads[1] : p.heads[0];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int h = h0 + RPW * i;
      if (in && h < heads) {
        raw[i][0] = *reinterpret_cast<const RT*>(x + h * p.D + ca);
        raw[i][1] = *reinterpret_cast<const RT*>(x + h * p.D + cb);
      } else {
        raw[i][0] = raw[i][1] = RT{};
      }
    }
  };
  float w[8];
  int w_of = -1;
  if (hb < nb) load(hb);
  while (hb < nb) {
    const int s = hb >= p.blocks[0] ? 1 : 0, h0 = (hb - (s ? p.blocks[0] : 0)) * (RPW * NB) + sub;
    RT now[NB][2];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      now[i][0] = raw[i][0];
      now[i][1] = raw[i][1];
    }
    hb += (int)p.parts;
    if (hb < nb) load(hb);
    const float* wp = s ? p.w[1] : p.w[0];
    if (s != w_of) {
      w_of = s;
      if (wp && in) {
        unpack4<F32>(wp + ca, &w[0]);
        unpack4<F32>(wp + cb, &w[4]);
      }
    }
    TO* y = reinterpret_cast<TO*>(s ? p.y[1] : p.y[0]) + t * (s ? p.ldy[1] : p.ldy[0]);
    const int heads = s ? p.heads[1] : p.heads[0];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      float u[8];
      unpack4<EI>(&now[i][0], &u[0]);
      unpack4<EI>(&now[i][1], &u[4]);
      if (wp) {
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(u[k], u[k], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = u[k] * r * w[k];
      }
      if (turns) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int a = INTERLEAVED ? 2 * k : k, c = INTERLEAVED ? 2 * k + 1 : k + 4;
          const float x = u[a], z = u[c];
          u[a] = fmaf(x, cs[k], -z * sn[k]);
          u[c] = fmaf(z, cs[k], x * sn[k]);
        }
      }
      const int h = h0 + RPW * i;
      if (in && h < heads) {
        pack4<EO>(y + h * p.D + ca, &u[0]);
        pack4<EO>(y + h * p.D + cb, &u[4]);
      }
    }
  }
}

}  // namespace qkr

gptq_status qk_norm_rope_launch(const void* Q, const void* K, int in_dtype, long long T, int hq, int hk, int D,
                                long long ldq, long long ldk, const float* wq, const float* wk, float eps,
                                const float* cosv, const float* sinv, long long n_pos, int rot, int interleaved,
                                const int* positions, void* Qo, void* Ko, int out_dtype, long long ldqo,
                                long long ldko, cudaStream_t s) {
  using namespace qkr;
  Params p{};
  p.x[0] = Q; p.x[1] = K; p.y[0] = Qo; p.y[1] = Ko; p.w[0] = wq; p.w[1] = wk;
  p.ldx[0] = ldq; p.ldx[1] = ldk; p.ldy[0] = ldqo; p.ldy[1] = ldko;
  p.heads[0] = hq; p.heads[1] = hk;
  p.T = (uint32_t)T; p.D = D; p.rot = rot; p.eps = eps;
  p.cosv = cosv; p.sinv = sinv; p.pos = positions; p.n_pos = n_pos;
  const int rows = (32 / lanes_per_row(D)) * NB;
  for (int k = 0; k < 2; ++k) p.blocks[k] = (p.heads[k] + rows - 1) / rows;
  // a warp per token where that alone fills the GPU twice over, else as many as there are blocks
  const long long nb = p.blocks[0] + p.blocks[1], fill = 32LL * sm_count();
  p.parts = (uint32_t)std::min(nb, std::max(1LL, (fill + T - 1) / T));
  const unsigned long long units = (unsigned long long)T * p.parts;
  if (units > 0xFFFFFFFFull - WARPS) return set_error(GPTQ_ERR_INVALID_ARG, "too many rows for one launch");
  const unsigned grid = (unsigned)((units + WARPS - 1) / WARPS);
  with_dtype(in_dtype, [&](auto ei) {
    with_dtype(out_dtype, [&](auto eo) {
      with_lanes(D, [&](auto lpr) {
        constexpr int LPR = decltype(lpr)::value;
        if (interleaved)
          qk_norm_rope_kernel<decltype(ei), decltype(eo), LPR, true><<<grid, WARPS * 32, 0, s>>>(p, device_error_word());
        else
          qk_norm_rope_kernel<decltype(ei), decltype(eo), LPR, false><<<grid, WARPS * 32, 0, s>>>(p, device_error_word());
      });
    });
  });
  count_launch();
  return check_launch("qk_norm_rope_kernel");
}

}  // namespace gptq
