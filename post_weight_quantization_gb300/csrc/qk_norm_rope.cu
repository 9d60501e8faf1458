// The RMS norm of every query and key head and the position rotation, in one pass.
//
//   n = x * rsqrt(mean(x^2) + eps) * w,   then every pair (n_i, n_j) turned by the angle of
//   its position: (n_i c - n_j s, n_j c + n_i s)
//
// A row (one head of one token) lies in LPR lanes, eight values each, so a row is one
// 16-byte load per lane (two for fp32) and the mean is log2(LPR) shuffles. The partner of
// a half-split pair is rot/2 values away, a whole number of lanes (rot % 16 == 0): it
// comes by shuffle. Arithmetic is fp32; the one rounding is the store.
//
// Bound: HBM bandwidth (every value read once and written once).
#include <type_traits>

#include "elem.cuh"

namespace gptq {
namespace qkr {

constexpr int WARPS = 4;

struct Params {
  const void* x[2];            // Q, K
  void* y[2];
  const float* w[2];
  long long ldx[2], ldy[2];
  int heads[2];
  int blocks[2];               // head blocks per token
  long long T;
  int D, rot, interleaved;
  float eps;
  const float* cosv;
  const float* sinv;
  const int* pos;
  long long n_pos;
};

// One warp: NB head rows per lane group of one token's head block, so the token's cosines
// and sines are read once for NB rows.
template <typename EI, typename EO, int LPR, int NB>
__global__ void __launch_bounds__(WARPS * 32) qk_norm_rope_kernel(Params p, int* __restrict__ err) {
  constexpr int RPW = 32 / LPR;                       // rows per warp at once
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR, c = 8 * l;
  const long long unit = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
  const int per_token = p.blocks[0] + p.blocks[1];
  const long long t = unit / per_token;
  if (t >= p.T) return;
  int hb = (int)(unit - t * per_token);
  const int s = hb >= p.blocks[0] ? 1 : 0;
  if (s) hb -= p.blocks[0];
  const bool in = c < p.D;
  const int h0 = hb * (RPW * NB) + sub;
  const typename EI::T* x = reinterpret_cast<const typename EI::T*>(p.x[s]) + t * p.ldx[s] + c;
  typename EO::T* y = reinterpret_cast<typename EO::T*>(p.y[s]) + t * p.ldy[s] + c;

  float v[NB][8];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int h = h0 + b * RPW;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[b][k] = 0.0f;
    if (in && h < p.heads[s]) unpack8<EI>(x + (long long)h * p.D, v[b]);
  }
  float cv[8], sv[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) { cv[k] = 1.0f; sv[k] = 0.0f; }
  const int half = p.rot >> 1;
  if (p.rot) {
    const int pos = p.pos[t];
    if (pos < 0 || pos >= p.n_pos) {
      if (lane == 0) report_device_error(err, DEVERR_INDEX);
    } else if (c < p.rot) {
      if (p.interleaved) {                            // pairs (2i, 2i + 1): four angles a lane
        const float4 a = *reinterpret_cast<const float4*>(p.cosv + (long long)pos * half + (c >> 1));
        const float4 b = *reinterpret_cast<const float4*>(p.sinv + (long long)pos * half + (c >> 1));
        cv[0] = cv[1] = a.x; cv[2] = cv[3] = a.y; cv[4] = cv[5] = a.z; cv[6] = cv[7] = a.w;
        sv[0] = -b.x; sv[1] = b.x; sv[2] = -b.y; sv[3] = b.y;
        sv[4] = -b.z; sv[5] = b.z; sv[6] = -b.w; sv[7] = b.w;
      } else {
        const bool low = c < half;
        const long long o = (long long)pos * half + (low ? c : c - half);
        unpack8<F32>(p.cosv + o, cv);
        unpack8<F32>(p.sinv + o, sv);
        if (low) {
#pragma unroll
          for (int k = 0; k < 8; ++k) sv[k] = -sv[k];
        }
      }
    }
  }
  float w[8];
  const float* wp = p.w[s];
  if (wp && in) unpack8<F32>(wp + c, w);
  const int partner = (c < half) ? lane + half / 8 : (c < p.rot ? lane - half / 8 : lane);
  const float inv_d = 1.0f / (float)p.D;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (wp) {
      float ss = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[b][k], v[b][k], ss);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = 1.0f / sqrtf(fmaf(ss, inv_d, p.eps));
      if (in) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[b][k] = v[b][k] * r * w[k];
      }
    }
    if (p.rot) {
      float o[8];
      if (p.interleaved) {
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = v[b][k ^ 1];
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = __shfl_sync(0xffffffffu, v[b][k], partner);
      }
      if (c < p.rot) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[b][k] = fmaf(v[b][k], cv[k], o[k] * sv[k]);
      }
    }
    const int h = h0 + b * RPW;
    if (in && h < p.heads[s]) pack8<EO>(y + (long long)h * p.D, v[b]);
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
  p.T = T; p.D = D; p.rot = rot; p.interleaved = interleaved; p.eps = eps;
  p.cosv = cosv; p.sinv = sinv; p.pos = positions; p.n_pos = n_pos;
  long long grid = 0;
  bool fits = true;
  with_dtype(in_dtype, [&](auto ei) {
    with_dtype(out_dtype, [&](auto eo) {
      with_lanes(D, [&](auto lpr) {
        constexpr int LPR = decltype(lpr)::value, NB = 4, RPW = 32 / LPR;
        for (int k = 0; k < 2; ++k) p.blocks[k] = (p.heads[k] + RPW * NB - 1) / (RPW * NB);
        grid = (T * (p.blocks[0] + p.blocks[1]) + WARPS - 1) / WARPS;
        if (grid > 0x7FFFFFFFLL) { fits = false; return; }
        qk_norm_rope_kernel<decltype(ei), decltype(eo), LPR, NB>
            <<<(unsigned)grid, WARPS * 32, 0, s>>>(p, device_error_word());
      });
    });
  });
  if (!fits) return set_error(GPTQ_ERR_INVALID_ARG, "too many rows for one launch");
  count_launch();
  return check_launch("qk_norm_rope_kernel");
}

}  // namespace gptq
