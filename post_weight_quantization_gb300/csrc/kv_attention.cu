// Attention over the 4-bit paged cache.
//
//   o_i = sum_j p_ij v_j,   p_i = softmax over the seen j of sm_scale * q_i . k_j,
//   k_j = code * scale_j + low_j (and v_j alike), one (scale, low) per token and head
//
// One warp per query token and head: a lane holds D / 32 values of q and of the running
// output, the scores' maximum and sum run along (one pass over the cache), everything fp32.
#include <math_constants.h>

#include <type_traits>

#include "elem.cuh"

namespace gptq {
namespace kva {

constexpr int WARPS = 4;

struct Params {
  const void* Q;
  void* O;
  float* lse;
  const int* cu_q;
  const int* kv_lens;
  const int* table;
  const uint8_t* pool;
  long long ldq, ldo, ldt, total_q, table_width, num_pages;
  int Hq, H, page, batch, causal;
  long long window;
  float scale_log2;            // sm_scale * log2(e)
};

template <typename E, int D>
__global__ void __launch_bounds__(WARPS * 32) kv_attention_kernel(Params p, int* __restrict__ err) {
  constexpr int VPL = D / 32;                            // values per lane
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
  const long long tok = unit / p.Hq;
  if (tok >= p.total_q) return;
  const int hq = (int)(unit - tok * p.Hq), h = hq / (p.Hq / p.H);
  int lo = 0, hi = p.batch;                              // the last sequence that starts at or before tok
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu_q[mid] <= tok) lo = mid; else hi = mid - 1;
  }
  const int b = lo;
  if (b >= p.batch || tok < p.cu_q[0]) return;
  const long long nq = (long long)p.cu_q[b + 1] - p.cu_q[b];
  long long len = p.kv_lens[b];
  if (len < 0 || len > p.table_width * p.page) {
    if (lane == 0) report_device_error(err, DEVERR_INDEX);
    len = len < 0 ? 0 : p.table_width * p.page;
  }
  const long long pos = len - nq + (tok - p.cu_q[b]);
  const long long end = p.causal ? (pos + 1 < len ? pos + 1 : len) : len;
  const long long begin = (p.window > 0 && pos - p.window + 1 > 0) ? pos - p.window + 1 : 0;
  float q[VPL], o[VPL];
  const typename E::T* qp = reinterpret_cast<const typename E::T*>(p.Q) + tok * p.ldq + (long long)hq * D + lane * VPL;
#pragma unroll
  for (int k = 0; k < VPL; ++k) { q[k] = (float)qp[k]; o[k] = 0.0f; }
  float m = -CUDART_INF_F, sum = 0.0f;
  const long long block = (long long)p.page * (D + 8);
  for (long long j = begin; j < end; ++j) {
    const int page = p.table[b * p.ldt + j / p.page], at = (int)(j % p.page);
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) report_device_error(err, DEVERR_INDEX);
      continue;
    }
    const uint8_t* blk = p.pool + ((long long)page * p.H + h) * block;
    const uint16_t* n = reinterpret_cast<const uint16_t*>(blk + (long long)p.page * D) + 4 * at;
    float num[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) num[k] = __half2float(__ushort_as_half(n[k]));
    const uint8_t* kc = blk + (long long)at * (D / 2) + lane * (VPL / 2);
    const uint8_t* vc = kc + (long long)p.page * (D / 2);
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < VPL / 2; ++k) {
      dot = fmaf(q[2 * k], fmaf((float)(kc[k] & 15), num[0], num[1]), dot);
      dot = fmaf(q[2 * k + 1], fmaf((float)(kc[k] >> 4), num[0], num[1]), dot);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
    const float x = dot * p.scale_log2, mn = fmaxf(m, x);
    const float f = mn == -CUDART_INF_F ? 0.0f : exp2f(m - mn), e = mn == -CUDART_INF_F ? 0.0f : exp2f(x - mn);
    m = mn;
    sum = fmaf(sum, f, e);
#pragma unroll
    for (int k = 0; k < VPL / 2; ++k) {
      o[2 * k] = fmaf(e, fmaf((float)(vc[k] & 15), num[2], num[3]), o[2 * k] * f);
      o[2 * k + 1] = fmaf(e, fmaf((float)(vc[k] >> 4), num[2], num[3]), o[2 * k + 1] * f);
    }
  }
  typename E::T* op = reinterpret_cast<typename E::T*>(p.O) + tok * p.ldo + (long long)hq * D + lane * VPL;
  const float inv = begin < end ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    float x = o[k] * inv;
    if (std::is_same<E, F16>::value && x == x) x = fminf(fmaxf(x, -65504.0f), 65504.0f);
    op[k] = (typename E::T)x;
  }
  if (p.lse && lane == 0) p.lse[tok * p.Hq + hq] = begin < end ? (m + log2f(sum)) * 0.6931471805599453f : -CUDART_INF_F;
}

}  // namespace kva

size_t kv_attention_workspace_bytes(long long, int, int, int, long long, long long) { return 256; }

gptq_status kv_attention_launch(const void* Q, int dtype, long long total_q, int Hq, int H, int D, long long ldq,
                                const int* cu_q, const int* kv_lens, const int* table, long long ldt,
                                long long table_width, long long batch, long long max_q, const void* pool,
                                long long num_pages, int page, float sm_scale, int causal, long long window, void* O,
                                long long ldo, float* lse, void* ws, cudaStream_t s) {
  using namespace kva;
  (void)ws;
  (void)max_q;
  Params p{};
  p.Q = Q; p.O = O; p.lse = lse; p.cu_q = cu_q; p.kv_lens = kv_lens; p.table = table;
  p.pool = reinterpret_cast<const uint8_t*>(pool);
  p.ldq = ldq; p.ldo = ldo; p.ldt = ldt; p.total_q = total_q; p.table_width = table_width; p.num_pages = num_pages;
  p.Hq = Hq; p.H = H; p.page = page; p.batch = (int)batch; p.causal = causal; p.window = window;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  const long long grid = (total_q * Hq + WARPS - 1) / WARPS;
  if (grid > 0x7FFFFFFFLL) return set_error(GPTQ_ERR_INVALID_ARG, "too many query heads for one launch");
  auto go = [&](auto e, auto d) {
    kv_attention_kernel<decltype(e), decltype(d)::value><<<(unsigned)grid, WARPS * 32, 0, s>>>(p, device_error_word());
  };
  auto width = [&](auto e) {
    if (D == 64) go(e, std::integral_constant<int, 64>{});
    else if (D == 128) go(e, std::integral_constant<int, 128>{});
    else go(e, std::integral_constant<int, 256>{});
  };
  if (dtype == GPTQ_BF16) width(BF16{}); else width(F16{});
  count_launch();
  return check_launch("kv_attention_kernel");
}

}  // namespace gptq
