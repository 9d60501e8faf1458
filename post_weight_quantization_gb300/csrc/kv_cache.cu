// Rows of the 4-bit paged cache: K and V rows quantized into their pages, and read back.
//
//   low = fp16(min x), scale = fp16((max x - min x) / 15),
//   code = clamp(round((x - low) / scale), 0, 15),   value = code * scale + low
//
// One page of one head is one block: K codes of its page_size tokens, V codes, then four
// fp16 per token (K scale, K low, V scale, V low), so attention fetches a page of a head
// with one contiguous copy. A row (K or V of one token and head) lies in LPR = D / 8
// lanes, eight values each: one 16-byte load and one word of eight codes per lane.
//
// The division is exact to the last bit without a division per value: with
// r = fl(1 / scale), q = fl(a r), q' = fl(q + fl(a - q scale) r) is the correctly rounded
// a / scale (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990), and a is limited to [0, 15 scale] first, which limits the quotient
// to [0, 15] exactly and keeps infinities out.
//
// Bound: HBM bandwidth (16-bit rows read once, D / 2 + 4 bytes written per row).
#include <type_traits>

#include "elem.cuh"

namespace gptq {
namespace kvc {

constexpr int WARPS = 4;
constexpr float kHalfMax = 65504.0f;

__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

struct Params {
  const void* x[2];            // K, V
  long long ldx[2];
  void* y[2];                  // read back
  long long ldy[2];
  const long long* slots;
  uint8_t* pool;
  long long T, n_slots;        // tokens, num_pages * page_size
  int H, page;
};

template <int LPR>
__device__ __forceinline__ uint8_t* block_of(const Params& p, long long slot, int h, int& at) {
  constexpr int D = 8 * LPR;
  const long long page = slot / p.page;
  at = (int)(slot - page * p.page);
  return p.pool + (page * p.H + h) * ((long long)p.page * (D + 8));
}

// Row r of the call: r = (token * H + head) * 2 + (0: K, 1: V).
template <typename E, int LPR>
__global__ void __launch_bounds__(WARPS * 32) kv_append_kernel(Params p, int* __restrict__ err) {
  constexpr int D = 8 * LPR, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR;
  const long long r = ((long long)blockIdx.x * WARPS + (threadIdx.x >> 5)) * RPW + lane / LPR;
  const long long th = r >> 1;
  const long long t = th / p.H;
  const int h = (int)(th - t * p.H), kv = (int)(r & 1);
  bool live = t < p.T;
  const long long slot = live ? p.slots[t] : -1;
  if (slot >= p.n_slots && l == 0) report_device_error(err, DEVERR_INDEX);
  live = slot >= 0 && slot < p.n_slots;
  float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (live) unpack8<E>(reinterpret_cast<const typename E::T*>(p.x[kv]) + t * p.ldx[kv] + (long long)h * D + 8 * l, v);
  float lo = v[0], hi = v[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) { lo = min_nan(lo, v[k]); hi = max_nan(hi, v[k]); }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const bool bad = lo != lo;
  lo = bad ? 0.0f : fminf(fmaxf(lo, -kHalfMax), kHalfMax);     // a NaN row: codes of 0, its scale says the rest
  hi = bad ? 0.0f : fminf(fmaxf(hi, -kHalfMax), kHalfMax);
  const __half hs = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f)), hl = __float2half_rn(lo);
  const float sc = __half2float(hs), low = __half2float(hl);
  const float inv = sc > 0.0f ? __frcp_rn(sc) : 0.0f, top = 15.0f * sc;
  uint32_t word = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float a = fminf(fmaxf(__fsub_rn(v[k], low), 0.0f), top);
    float q = __fmul_rn(a, inv);
    q = __fmaf_rn(__fmaf_rn(-q, sc, a), inv, q);
    // 2^23 + q rounds q to an integer, ties to even, in the mantissa's low bits
    word |= (__float_as_uint(__fadd_rn(q, 8388608.0f)) & 15u) << (4 * k);
  }
  if (!live) return;
  int at;
  uint8_t* b = block_of<LPR>(p, slot, h, at);
  reinterpret_cast<uint32_t*>(b + ((long long)kv * p.page + at) * (D / 2))[l] = word;
  if (l == 0) {
    const uint32_t s16 = bad ? 0x7FFFu : (uint32_t)__half_as_ushort(hs);
    reinterpret_cast<uint32_t*>(b + (long long)p.page * D)[2 * at + kv] = s16 | ((uint32_t)__half_as_ushort(hl) << 16);
  }
}

template <typename E, int LPR>
__global__ void __launch_bounds__(WARPS * 32) kv_read_kernel(Params p, int* __restrict__ err) {
  constexpr int D = 8 * LPR, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR;
  const long long r = ((long long)blockIdx.x * WARPS + (threadIdx.x >> 5)) * RPW + lane / LPR;
  const long long th = r >> 1;
  const long long t = th / p.H;
  const int h = (int)(th - t * p.H), kv = (int)(r & 1);
  if (t >= p.T) return;
  const long long slot = p.slots[t];
  float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (slot >= p.n_slots) {
    if (l == 0) report_device_error(err, DEVERR_INDEX);
  } else if (slot >= 0) {
    int at;
    const uint8_t* b = block_of<LPR>(p, slot, h, at);
    const uint32_t word = reinterpret_cast<const uint32_t*>(b + ((long long)kv * p.page + at) * (D / 2))[l];
    const uint32_t n = reinterpret_cast<const uint32_t*>(b + (long long)p.page * D)[2 * at + kv];
    const float sc = __half2float(__ushort_as_half((unsigned short)n));
    const float low = __half2float(__ushort_as_half((unsigned short)(n >> 16)));
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = fmaf((float)((word >> (4 * k)) & 15u), sc, low);
    if (std::is_same<E, F16>::value) {                  // 15 scale + low can round past fp16's range
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (v[k] == v[k]) v[k] = fminf(fmaxf(v[k], -kHalfMax), kHalfMax);
    }
  }
  pack8<E>(reinterpret_cast<typename E::T*>(p.y[kv]) + t * p.ldy[kv] + (long long)h * D + 8 * l, v);
}

template <typename F>
void with_width(int D, F&& f) {
  if (D == 64) f(std::integral_constant<int, 8>{});
  else if (D == 128) f(std::integral_constant<int, 16>{});
  else f(std::integral_constant<int, 32>{});
}

}  // namespace kvc

gptq_status kv_append_launch(const void* K, const void* V, int dtype, long long T, int H, int D, long long ldk,
                             long long ldv, const long long* slots, void* pool, long long num_pages, int page,
                             cudaStream_t s) {
  using namespace kvc;
  Params p{};
  p.x[0] = K; p.x[1] = V; p.ldx[0] = ldk; p.ldx[1] = ldv;
  p.slots = slots; p.pool = reinterpret_cast<uint8_t*>(pool);
  p.T = T; p.n_slots = num_pages * page; p.H = H; p.page = page;
  const long long rows = 2 * T * H, per = WARPS * (32 / (D / 8)), grid = (rows + per - 1) / per;
  if (grid > 0x7FFFFFFFLL) return set_error(GPTQ_ERR_INVALID_ARG, "too many rows for one launch");
  with_dtype(dtype, [&](auto e) {
    with_width(D, [&](auto lpr) {
      kv_append_kernel<decltype(e), decltype(lpr)::value>
          <<<(unsigned)grid, WARPS * 32, 0, s>>>(p, device_error_word());
    });
  });
  count_launch();
  return check_launch("kv_append_kernel");
}

gptq_status kv_read_launch(const void* pool, long long num_pages, int page, int H, int D, const long long* slots,
                           long long T, void* K, void* V, int dtype, long long ldk, long long ldv, cudaStream_t s) {
  using namespace kvc;
  Params p{};
  p.y[0] = K; p.y[1] = V; p.ldy[0] = ldk; p.ldy[1] = ldv;
  p.slots = slots; p.pool = reinterpret_cast<uint8_t*>(const_cast<void*>(pool));
  p.T = T; p.n_slots = num_pages * page; p.H = H; p.page = page;
  const long long rows = 2 * T * H, per = WARPS * (32 / (D / 8)), grid = (rows + per - 1) / per;
  if (grid > 0x7FFFFFFFLL) return set_error(GPTQ_ERR_INVALID_ARG, "too many rows for one launch");
  with_dtype(dtype, [&](auto e) {
    with_width(D, [&](auto lpr) {
      kv_read_kernel<decltype(e), decltype(lpr)::value><<<(unsigned)grid, WARPS * 32, 0, s>>>(p, device_error_word());
    });
  });
  count_launch();
  return check_launch("kv_read_kernel");
}

}  // namespace gptq
