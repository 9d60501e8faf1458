// A packed projection with the low-rank adapters of many requests beside it:
//
//   Y[t] = X[t] W_hat^T + alpha[a] (X[t] A[a]^T) B[a]^T,   a = ids[t]
//
// adapter_shrink_kernel  U[t][r] = alpha[a] * A[a][r] . X[t] (fp32, workspace): one CTA per
//                        token, its warps over the ranks
// base                   X W_hat^T in fp32: the dequant GEMV or GEMM
// adapter_expand_kernel  Y[t][i] = base + B[a][i] . U[t]
#include <algorithm>

#include "elem.cuh"

namespace gptq {

gptq_status dequant_gemv_launch(const uint32_t* qweight, const float* scales, const float* zeros, const int32_t* g_idx,
                                long long m, long long d, int bits, int group_size, const uint16_t* X, long long T,
                                long long ldx, float* Y, long long ldy, cudaStream_t s);
size_t dequant_gemm_workspace_bytes(long long m, long long d);
gptq_status dequant_gemm_launch(const uint32_t* qweight, const float* scales, const float* zeros, long long m,
                                long long d, int bits, int group_size, const uint16_t* X, long long T, long long ldx,
                                void* Y, int y_bf16, long long ldy, void* ws, cudaStream_t s);

namespace adp {

constexpr int WARPS = 8;

__global__ void __launch_bounds__(WARPS * 32)
adapter_shrink_kernel(const uint16_t* __restrict__ X, long long ldx, int d, const uint16_t* __restrict__ A,
                      const float* __restrict__ alpha, long long n_adapters, int rank, const int* __restrict__ ids,
                      float* __restrict__ U, int* __restrict__ err) {
  const long long t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int a = ids[t];
  if (a >= n_adapters && threadIdx.x == 0) report_device_error(err, DEVERR_INDEX);
  const bool has = a >= 0 && a < n_adapters;
  for (int r = warp; r < rank; r += WARPS) {
    float sum = 0.0f;
    if (has) {
      const uint16_t* ar = A + ((long long)a * rank + r) * d;
      for (int c = 8 * lane; c < d; c += 256) {
        float x[8], w[8];
        unpack8<BF16>(X + t * ldx + c, x);
        unpack8<BF16>(ar + c, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum = fmaf(x[k], w[k], sum);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (alpha) sum *= alpha[a];
    }
    if (lane == 0) U[t * rank + r] = sum;
  }
}

__global__ void __launch_bounds__(256)
adapter_expand_kernel(const float* __restrict__ base, long long ldb, const uint16_t* __restrict__ B,
                      long long n_adapters, int rank, const int* __restrict__ ids, const float* __restrict__ U,
                      long long T, long long m, void* Y, int y_bf16, long long ldy) {
  const long long n = T * m;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const long long t = i / m, r = i - t * m;
    float sum = base[t * ldb + r];
    const int a = ids ? ids[t] : -1;
    if (a >= 0 && a < n_adapters) {
      const uint16_t* b = B + ((long long)a * m + r) * rank;
      const float* u = U + t * rank;
      for (int c = 0; c < rank; c += 8) {
        float w[8];
        unpack8<BF16>(b + c, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum = fmaf(w[k], u[c + k], sum);
      }
    }
    if (y_bf16) reinterpret_cast<__nv_bfloat16*>(Y)[t * ldy + r] = __float2bfloat16_rn(sum);
    else reinterpret_cast<float*>(Y)[t * ldy + r] = sum;
  }
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace adp

// Workspace: U (T x rank fp32), the base product (T x m fp32), the dequant GEMM's operand.
size_t adapter_workspace_bytes(long long m, long long d, int bits, int group_size, long long T, int rank) {
  using namespace adp;
  (void)bits;
  (void)group_size;
  return round256(4 * (size_t)T * rank) + round256(4 * (size_t)T * m) + dequant_gemm_workspace_bytes(m, d) + 256;
}

gptq_status adapter_linear_launch(const uint32_t* qweight, const float* scales, const float* zeros, long long m,
                                  long long d, int bits, int group_size, const uint16_t* X, long long T, long long ldx,
                                  const uint16_t* A, const uint16_t* B, const float* alpha, long long n_adapters,
                                  int rank, const int* ids, void* Y, int y_dtype, long long ldy, void* ws,
                                  cudaStream_t s) {
  using namespace adp;
  float* U = reinterpret_cast<float*>(ws);
  float* base = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + round256(4 * (size_t)T * rank));
  void* gws = reinterpret_cast<uint8_t*>(base) + round256(4 * (size_t)T * m);
  if (ids) {
    adapter_shrink_kernel<<<(unsigned)T, WARPS * 32, 0, s>>>(X, ldx, (int)d, A, alpha, n_adapters, rank, ids, U,
                                                            device_error_word());
    count_launch();
    if (gptq_status st = check_launch("adapter_shrink_kernel")) return st;
  }
  gptq_status st = T <= 32 ? dequant_gemv_launch(qweight, scales, zeros, nullptr, m, d, bits, group_size, X, T, ldx, base, m, s)
                           : dequant_gemm_launch(qweight, scales, zeros, m, d, bits, group_size, X, T, ldx, base, 0, m, gws, s);
  if (st) return st;
  const long long grid = std::min<long long>((T * m + 255) / 256, 16LL * sm_count());
  adapter_expand_kernel<<<(unsigned)grid, 256, 0, s>>>(base, m, B, n_adapters, rank, ids, U, T, m, Y,
                                                       y_dtype == GPTQ_BF16, ldy);
  count_launch();
  return check_launch("adapter_expand_kernel");
}

}  // namespace gptq
