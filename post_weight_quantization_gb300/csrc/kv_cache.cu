// Rows of the 4-bit paged cache: K and V rows quantized into their pages, and read back.
//
//   low = fp16(min x), scale = fp16((max x - min x) / 15),
//   code = clamp(round((x - low) / scale), 0, 15),   value = code * scale + low
//
// One page of one head is one block: K codes of its page_size tokens, V codes, then four
// fp16 per token (K scale, K low, V scale, V low), so attention fetches a page of a head
// with one contiguous copy.
//
// The divisions are exact to the last bit without the divide's instructions: with
// r = fl(1 / s), q = fl(a r), q' = fl(q + fl(a - q s) r) is the correctly rounded
// a / s (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990); code_of has the limits.
//
// Bound: HBM bandwidth (16-bit rows read once, D / 2 + 4 bytes written per row). Measured, 30011 tokens
// of 8 heads of 128: appended in 30 us, read back in 24 us (4.85 TB/s over both, 72 % of a plain copy's
// rate); instruction issue is next (72 % and 55 % busy).
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

__device__ __forceinline__ float2 to_float2(__half2 h) { return __half22float2(h); }
__device__ __forceinline__ float2 to_float2(__nv_bfloat162 h) { return __bfloat1622float2(h); }
__device__ __forceinline__ __half2 lows_of(__half2 a, __half2 b) { return __lows2half2(a, b); }
__device__ __forceinline__ __half2 highs_of(__half2 a, __half2 b) { return __highs2half2(a, b); }
__device__ __forceinline__ __nv_bfloat162 lows_of(__nv_bfloat162 a, __nv_bfloat162 b) { return __lows2bfloat162(a, b); }
__device__ __forceinline__ __nv_bfloat162 highs_of(__nv_bfloat162 a, __nv_bfloat162 b) { return __highs2bfloat162(a, b); }

// a / s, correctly rounded, with inv = fl(1 / s).
__device__ __forceinline__ float divide(float a, float s, float inv) {
  const float q = __fmul_rn(a, inv);
  return __fmaf_rn(__fmaf_rn(-q, s, a), inv, q);
}
// fl(1 / s) of an fp16 value: the hardware's approximation and one Newton step (the GPU tests have every
// scale that a row can have, with values on and next to the ties between codes).
__device__ __forceinline__ float reciprocal(float s) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  return __fmaf_rn(__fmaf_rn(-s, y, 1.0f), y, y);
}

// Sixteen values of a row as they lie in memory: eight at 8 l and eight at D / 2 + 8 l of lane l.
template <typename E> struct alignas(16) Row8 { uint32_t w[4]; };
template <> struct alignas(16) Row8<F32> { uint32_t w[8]; };
template <typename E> struct Row16 { Row8<E> r[2]; };

// Smallest and largest value of a row (NaN if it holds one) over its LANES lanes: pairs at a
// time for the 16-bit types, the lanes' (minimum, -maximum) as one pair.
template <typename E, int LANES>
__device__ __forceinline__ void row_range(const Row16<E>& r, float& lo, float& hi) {
  if constexpr (std::is_same<E, F32>::value) {
    lo = hi = __uint_as_float(r.r[0].w[0]);
#pragma unroll
    for (int k = 1; k < 16; ++k) {
      const float v = __uint_as_float(r.r[k >> 3].w[k & 7]);
      lo = min_nan(lo, v);
      hi = max_nan(hi, v);
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
  } else {
    using P = typename std::conditional<std::is_same<E, BF16>::value, __nv_bfloat162, __half2>::type;
    const P *p = reinterpret_cast<const P*>(r.r[0].w), *q = reinterpret_cast<const P*>(r.r[1].w);
    P mn = __hmin2_nan(p[0], q[0]), mx = __hmax2_nan(p[0], q[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) {
      mn = __hmin2_nan(mn, __hmin2_nan(p[k], q[k]));
      mx = __hmax2_nan(mx, __hmax2_nan(p[k], q[k]));
    }
    mx = __hneg2(mx);
    P both = __hmin2_nan(lows_of(mn, mx), highs_of(mn, mx));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      uint32_t w = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t*>(&both), o);
      both = __hmin2_nan(both, *reinterpret_cast<P*>(&w));
    }
    const float2 f = to_float2(both);
    lo = f.x;
    hi = -f.y;
  }
}

// Two fp32 values in one register pair: sum, product, multiply-add of both at once.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// The codes of eight values as a word: round((x - low) / s) limited to [0, 15], ties to even, in
// fp32. The limits are put on the numerator (15 s / s is 15 exactly, and an infinity stays out of
// the correction). Adding 1.5 * 2^23 rounds the quotient to an integer, which lies in the sum's low
// bits; the eight sums' other bits leave the word as one constant (mod 2^32).
__device__ __forceinline__ uint32_t codes_of(const float (&v)[8], float low, float s, float inv, float top) {
  const uint64_t low2 = pair(-low, -low), s2 = pair(-s, -s), inv2 = pair(inv, inv), magic = pair(12582912.0f, 12582912.0f);
  uint32_t word = 0u - 0x4B400000u * 0x11111111u;
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const float2 a = halves(add2(pair(v[k], v[k + 1]), low2));
    const uint64_t n = pair(fmaxf(fminf(a.x, top), 0.0f), fmaxf(fminf(a.y, top), 0.0f));
    const uint64_t q = mul2(n, inv2);                   // the two steps of divide()
    const float2 c = halves(add2(fma2(fma2(q, s2, n), inv2, q), magic));
    word += __float_as_uint(c.x) << (4 * k);
    word += __float_as_uint(c.y) << (4 * k + 4);
  }
  return word;
}

// A warp takes one token and NB * RPW / 2 heads of it (RPW rows at once): NB rows per lane
// group, whose loads are all in flight before the first is used (the token's slot and its
// page, a 64-bit multiply by a host-computed reciprocal instead of a division, are the same
// for all of them). A lane holds 16 values of a row, and always of K or always of V, so that what is
// computed per row costs half as much as with eight and addresses are steps: the kernels are bound
// by instruction issue before bandwidth. NB is 4 where the heads fill it, else 2.
template <int D> constexpr int row_lanes() { return D / 16; }

struct Params {
  const void* x[2];            // K, V
  long long ldx[2];
  void* y[2];                  // read back
  long long ldy[2];
  const long long* slots;
  uint8_t* pool;
  long long n_slots;           // num_pages * page_size
  unsigned long long page_inv; // ceil(2^64 / page_size): slot * page_size < 2^48, so the high word is exact
  uint32_t T, blocks;          // tokens, head blocks per token
  int H, page;
};

// The token and the first head of a warp's unit; false past the last token.
template <int HEADS>
__device__ __forceinline__ bool unit_of(const Params& p, uint32_t& t, int& h0) {
  const uint32_t unit = blockIdx.x * WARPS + (threadIdx.x >> 5);
  t = unit / p.blocks;
  h0 = (int)(unit - t * p.blocks) * HEADS;
  return t < p.T;
}

template <int D>
__device__ __forceinline__ uint8_t* page_of(const Params& p, long long slot, int& at) {
  const long long page = (long long)__umul64hi((unsigned long long)slot, p.page_inv);
  at = (int)(slot - page * p.page);
  return p.pool + page * p.H * ((long long)p.page * (D + 8));
}

template <typename E, int D, int NB>
__global__ void __launch_bounds__(WARPS * 32) kv_append_kernel(Params p, int* __restrict__ err) {
  constexpr int LANES = row_lanes<D>(), RPW = 32 / LANES;
  const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES, kv = sub & 1;
  uint32_t t;
  int h0;
  if (!unit_of<NB * RPW / 2>(p, t, h0)) return;
  const long long slot = p.slots[t];
  h0 += sub >> 1;                                       // this lane's heads: h0, h0 + RPW / 2, ...
  const typename E::T* x = reinterpret_cast<const typename E::T*>(kv ? p.x[1] : p.x[0]) + t * (kv ? p.ldx[1] : p.ldx[0]) +
                           h0 * D + 8 * l;
  Row16<E> raw[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    raw[i] = Row16<E>{};
    if (h0 + i * (RPW / 2) < p.H) {
      raw[i].r[0] = *reinterpret_cast<const Row8<E>*>(x + i * (RPW / 2) * D);
      raw[i].r[1] = *reinterpret_cast<const Row8<E>*>(x + i * (RPW / 2) * D + D / 2);
    }
  }
  if (slot < 0) return;
  if (slot >= p.n_slots) {
    if (lane == 0) report_device_error(err, DEVERR_INDEX);
    return;
  }
  int at;
  uint8_t* page = page_of<D>(p, slot, at);
  const long long block = (long long)p.page * (D + 8);
  uint8_t* codes = page + h0 * block + (kv * p.page + at) * (D / 2) + 4 * l;
  uint8_t* nums = page + h0 * block + p.page * D + 8 * at + 4 * kv;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    float lo, hi;
    row_range<E, LANES>(raw[i], lo, hi);
    const bool bad = lo != lo;
    lo = bad ? 0.0f : fminf(fmaxf(lo, -kHalfMax), kHalfMax);   // a NaN row: codes of 0, its scale says the rest
    hi = bad ? 0.0f : fminf(fmaxf(hi, -kHalfMax), kHalfMax);
    constexpr float kFifteenth = 1.0f / 15.0f;
    const __half hs = __float2half_rn(divide(__fsub_rn(hi, lo), 15.0f, kFifteenth)), hl = __float2half_rn(lo);
    const float sc = __half2float(hs), low = __half2float(hl);
    const float inv = sc > 0.0f ? reciprocal(sc) : 0.0f, top = 15.0f * sc;
    uint32_t word[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float v[8];
      unpack8<E>(&raw[i].r[y], v);
      word[y] = codes_of(v, low, sc, inv, top);
    }
    if (h0 + i * (RPW / 2) >= p.H) continue;
    uint32_t* c = reinterpret_cast<uint32_t*>(codes + i * (RPW / 2) * block);
    c[0] = word[0];
    c[D / 16] = word[1];
    if (l == 0) {
      const uint32_t s16 = bad ? 0x7FFFu : (uint32_t)__half_as_ushort(hs);
      *reinterpret_cast<uint32_t*>(nums + i * (RPW / 2) * block) = s16 | ((uint32_t)__half_as_ushort(hl) << 16);
    }
  }
}

// Eight codes of a word times scale plus low, one rounding each. A code masked out of its place k
// and put under the exponent of 2^23 is 2^23 + 16^k code as a float; less 2^23 it is 16^k code exactly,
// and times scale 16^-k the same product as code times scale.
__device__ __forceinline__ void values_of(uint32_t word, uint64_t s01, uint64_t s23, uint64_t low2, float (&v)[8]) {
  const uint64_t magic = pair(-8388608.0f, -8388608.0f);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const uint32_t w = word >> (k < 4 ? 0 : 16);
    const uint64_t c = pair(__uint_as_float((w & (15u << (4 * (k & 2)))) | 0x4B000000u),
                            __uint_as_float((w & (240u << (4 * (k & 2)))) | 0x4B000000u));
    const float2 f = halves(fma2(add2(c, magic), k & 2 ? s23 : s01, low2));
    v[k] = f.x;
    v[k + 1] = f.y;
  }
}

template <typename E, int D, int NB>
__global__ void __launch_bounds__(WARPS * 32) kv_read_kernel(Params p, int* __restrict__ err) {
  constexpr int LANES = row_lanes<D>(), RPW = 32 / LANES;
  const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES, kv = sub & 1;
  uint32_t t;
  int h0;
  if (!unit_of<NB * RPW / 2>(p, t, h0)) return;
  const long long slot = p.slots[t];
  h0 += sub >> 1;
  const bool live = slot >= 0 && slot < p.n_slots;
  if (slot >= p.n_slots && lane == 0) report_device_error(err, DEVERR_INDEX);
  int at = 0;
  const uint8_t* page = live ? page_of<D>(p, slot, at) : nullptr;
  const long long block = (long long)p.page * (D + 8);
  const uint8_t* codes = page + h0 * block + (kv * p.page + at) * (D / 2) + 4 * l;
  const uint8_t* nums = page + h0 * block + p.page * D + 8 * at + 4 * kv;
  uint32_t word[NB][2], num[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    word[i][0] = word[i][1] = num[i] = 0u;
    if (live && h0 + i * (RPW / 2) < p.H) {
      const uint32_t* c = reinterpret_cast<const uint32_t*>(codes + i * (RPW / 2) * block);
      word[i][0] = c[0];
      word[i][1] = c[D / 16];
      num[i] = *reinterpret_cast<const uint32_t*>(nums + i * (RPW / 2) * block);
    }
  }
  typename E::T* y = reinterpret_cast<typename E::T*>(kv ? p.y[1] : p.y[0]) + t * (kv ? p.ldy[1] : p.ldy[0]) + h0 * D + 8 * l;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    if (h0 + i * (RPW / 2) >= p.H) continue;
    const float sc = __half2float(__ushort_as_half((unsigned short)num[i]));
    const float low = __half2float(__ushort_as_half((unsigned short)(num[i] >> 16)));
    const uint64_t low2 = pair(low, low), s01 = pair(sc, sc * 0.0625f), s23 = mul2(s01, pair(0.00390625f, 0.00390625f));
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      float v[8];
      values_of(word[i][z], s01, s23, low2, v);
      if (std::is_same<E, F16>::value) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (v[k] == v[k]) v[k] = fminf(fmaxf(v[k], -kHalfMax), kHalfMax);    // 15 scale + low can round past it
      }
      pack8<E>(y + i * (RPW / 2) * D + z * (D / 2), v);
    }
  }
}

template <typename F>
void with_width(int D, F&& f) {
  if (D == 64) f(std::integral_constant<int, 64>{});
  else if (D == 128) f(std::integral_constant<int, 128>{});
  else f(std::integral_constant<int, 256>{});
}

// Rows per lane group of a warp: four where the token's 2 H rows fill them.
int rows_of(int H, int D) { return 2 * H >= 4 * (32 / (D / 16)) ? 4 : 2; }

// Fills in the sizes for warps of `heads` heads; returns the grid (0: too large).
unsigned set_sizes(Params& p, long long T, int H, int heads, long long num_pages, int page, const long long* slots,
                   void* pool) {
  p.slots = slots;
  p.pool = reinterpret_cast<uint8_t*>(pool);
  p.n_slots = num_pages * page;
  p.page_inv = ~0ULL / (unsigned)page + 1;             // page is no power of two, or one: ceil(2^64 / page) either way
  p.T = (uint32_t)T;
  p.blocks = (uint32_t)((H + heads - 1) / heads);
  p.H = H;
  p.page = page;
  const unsigned long long units = (unsigned long long)p.T * p.blocks;
  return units > 0xFFFFFFFFull - WARPS ? 0u : (unsigned)((units + WARPS - 1) / WARPS);
}

}  // namespace kvc

gptq_status kv_append_launch(const void* K, const void* V, int dtype, long long T, int H, int D, long long ldk,
                             long long ldv, const long long* slots, void* pool, long long num_pages, int page,
                             cudaStream_t s) {
  using namespace kvc;
  Params p{};
  p.x[0] = K; p.x[1] = V; p.ldx[0] = ldk; p.ldx[1] = ldv;
  const int nb = rows_of(H, D);
  const unsigned grid = set_sizes(p, T, H, nb * (32 / (D / 16)) / 2, num_pages, page, slots, pool);
  if (!grid) return set_error(GPTQ_ERR_INVALID_ARG, "too many rows for one launch");
  with_dtype(dtype, [&](auto e) {
    with_width(D, [&](auto d) {
      if (nb == 4) kv_append_kernel<decltype(e), decltype(d)::value, 4><<<grid, WARPS * 32, 0, s>>>(p, device_error_word());
      else kv_append_kernel<decltype(e), decltype(d)::value, 2><<<grid, WARPS * 32, 0, s>>>(p, device_error_word());
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
  const int nb = rows_of(H, D);
  const unsigned grid = set_sizes(p, T, H, nb * (32 / (D / 16)) / 2, num_pages, page, slots, const_cast<void*>(pool));
  if (!grid) return set_error(GPTQ_ERR_INVALID_ARG, "too many rows for one launch");
  with_dtype(dtype, [&](auto e) {
    with_width(D, [&](auto d) {
      if (nb == 4) kv_read_kernel<decltype(e), decltype(d)::value, 4><<<grid, WARPS * 32, 0, s>>>(p, device_error_word());
      else kv_read_kernel<decltype(e), decltype(d)::value, 2><<<grid, WARPS * 32, 0, s>>>(p, device_error_word());
    });
  });
  count_launch();
  return check_launch("kv_read_kernel");
}

}  // namespace gptq
