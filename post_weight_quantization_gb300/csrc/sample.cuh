// The next token of each row of logits, from one given random number per row:
//
//   w_i = exp((l_i - max l) / temperature)
//   kept: the top_k largest logits; of those the ones before which, by falling logit, less than
//         top_p of the kept mass lies; of those the ones with w_i >= min_p. The lower index is the
//         larger of two equal logits. The largest is always kept.
//   token: the first kept i, by index, with w_0 + ... + w_i > u * (the kept mass)
//
// A row belongs to a cluster of CTAs and lies in their registers, so the logits are read once. A warp holds
// consecutive vectors of eight values, lane by lane, so the order of indexes is that of CTA, warp, vector,
// lane and value.
//
// The draw compares two sums of up to 2^18 terms, and one border among as many has to come out right: weights
// with the 2^-24 of fp32 would move a border of a flat row by a hundredth of a token's share. So
// the exponent is carried as two fp32 numbers, 2^y comes from a table of 2048 roots of two (32 bits)
// and a polynomial of second degree in the rest (2^-33), and the sums are integers in units of
// 2^-44, which no order of summation changes. FP64 would do it too, at 2 lanes an SM.
//
// Where few are kept (top_k up to 512, or little mass) they are listed, sorted and drawn from by one CTA. Otherwise
// top_k and top_p look for the logit where a count, or a mass, is reached. For a count the bits of an order-preserving integer of
// the logit are fixed five at a time, from the top: each thread adds its values to a column of 32 bins of its own in shared memory
// (no atomics, no conflicts); the columns' sums meet in the cluster through shared memory, and every warp finds the bin
// in which the sum is reached. Masses are the draw's integers, so that a border of top_p is the same however a row is split. A weight
// costs as much as seven comparisons, so fewer rounds weigh many values: the first bits are those of the distance to the
// largest logit, which part a row more evenly than the integer's, whose bits only part the values that share those. (256 rows of
// 151665 with top_p alone 894 us, with the integer's bits throughout 1078.)
//
// Bound: latency (a load, two or three exchanges of a cluster, a sort), and for large batches the phases of a CTA one after
// another. Measured: one row of 32000 12 us, 48 rows of 128256 with top_k, top_p and min_p 35 us, 256 rows of 151665 drawn
// whole 176 us (0.9 TB/s).
#pragma once

#include <math_constants.h>

#include <algorithm>
#include <array>
#include <type_traits>

#include "elem.cuh"

namespace gptq {
namespace smp {

constexpr int MOST = 8, WHOLE = 3, CUTS = 8;             // CTAs of a cluster at most; vectors a thread before a row gets more CTAs
constexpr int ROOTS = 2048, FRAC = 44;
constexpr int LIST = 2048, GUESS = 256;                  // candidates at most; how many where top_k does not say
constexpr int WIDE = 96, MASSES = 16;                    // words of a wide exchange, the first one of 32 masses in it
static_assert(MASSES + 64 < WIDE && MASSES % 2 == 0, "a wide exchange holds 32 masses and a word");
constexpr float T_MIN = 1e-30f, T_MAX = 1e30f;

// 2^(i / 2048) in units of 2^-31, from square roots by Newton's iteration.
constexpr double root(double x) {
  double r = 1.5;
  for (int k = 0; k < 8; ++k) r = 0.5 * (r + x / r);
  return r;
}
constexpr std::array<uint32_t, ROOTS> make_roots() {
  std::array<uint32_t, ROOTS> t{};
  double r[11] = {};
  double x = 2.0;
  for (int b = 10; b >= 0; --b) {                          // r[b] = 2^(2^b / 2048)
    x = root(x);
    r[b] = x;
  }
  for (int i = 0; i < ROOTS; ++i) {
    double v = 2147483648.0;
    for (int b = 0; b < 11; ++b)
      if (i >> b & 1) v *= r[b];
    t[i] = (uint32_t)(v + 0.5);
  }
  return t;
}
__device__ const std::array<uint32_t, ROOTS> d_roots = make_roots();

struct Params {
  const void* logits;
  long long ld;
  int V, vectors;              // 0: a row's vectors begin where 16-byte loads can, else this many from its first value on
  const float* u;
  const float* temperature;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  int* tokens;
  float* logprob;
};

// The candidates' part of `bins` while a row goes that way (and sorted, the weights of those that may be kept).
template <int NT>
struct Few {
  uint32_t keys[NT];           // largest key of each thread, sorted
  unsigned long long list[LIST];        // key and, falling, index: sorted, the order of top_k and top_p
  unsigned long long w[NT];
  unsigned long long sums[NT / 32];
};
struct Common {
  uint32_t roots[ROOTS];
  uint32_t part[WIDE];         // 32 words, or 16, 32 masses and one word
  uint32_t all[2][MOST][WIDE]; // the cluster's parts, two exchanges in turn
};
template <int NT, bool CUT>
struct Smem : Common {
  union {
    float bins[32][NT];        // a thread's column of counts
    uint32_t halves[2][32][NT / 2];    // two threads' column of masses, in two words
    Few<NT> few;
  };
};
template <int NT>
struct Smem<NT, false> : Common {};

__device__ __forceinline__ uint32_t key_of(float x) {      // grows with x; a NaN is the largest
  const uint32_t b = __float_as_uint(x);
  return x != x ? 0xFFFFFFFFu : b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }

// w of logit x in units of 2^-44: 2^(n + j / 2048) * 2^f with a root from the table and a polynomial.
__device__ __forceinline__ unsigned long long weight(const uint32_t* roots, float x, float big, float ch, float cl) {
  if (x == big) return 1ull << FRAC;
  // (x - big) * c as ph + pl
  const float d = x - big, t1 = d - x, e = (x - (d - t1)) + (-big - t1);
  const float ph = __fmul_rn(d, ch);                       // not contracted with what follows
  if (!(ph > -60.0f)) return 0;
  const float pl = fmaf(e, ch, fmaf(d, cl, fmaf(d, ch, -ph)));
  const float t = ph + 6144.0f;                            // to the nearest 2048th: 1.5 * 2^12 has that unit in the last place
  const int j = (int)__float_as_uint(t) - 0x45C00000;
  const float f = (ph - (t - 6144.0f)) + pl;
  const float q = f * fmaf(f, 0.240226507f, 0.693147181f); // 2^f - 1, |f| <= 2^-12
  const uint32_t r = roots[j & (ROOTS - 1)];
  const uint32_t m = r + (uint32_t)__mulhi((int)(r >> 1), __float2int_rn(q * 8589934592.0f));
  return ((unsigned long long)m << (FRAC - 31)) >> (-(j >> 11));
}

// Every CTA's 32 words (wide: all) of `part` to every CTA (all of which are known to run). Two buffers: one is written again only after all have read it and
// met once more.
struct Exchange {
  Common& s;
  int rank, n, warp, lane;
  uint32_t turn = 0;
  __device__ __forceinline__ const uint32_t (*operator()(bool wide = false))[WIDE] {
    __syncthreads();                                       // part is written
    const uint32_t b = turn++ & 1u;
    if (warp < n) {
      uint32_t to;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(&s.all[b][rank][lane])), "r"(warp));
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(s.part[lane]) : "memory");
      for (int i = 32; wide && i < WIDE; i += 32)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + 4 * i), "r"(s.part[i + lane]) : "memory");
    }
    __syncwarp();
    cluster_sync();
    return s.all[b];
  }
};

// The logit whose key has these leading bits: the others are zeros, or ones where a negative number's bits are inverted.
template <int SH>
__device__ __forceinline__ float of_lead(uint32_t lead) {
  const uint32_t k = lead << SH;
  return of_key(k >> 31 ? k : k | ((1u << SH) - 1u));
}

// log(w / total), w from the logit again: in units of 2^-44 a small one has few bits.
__device__ __forceinline__ float log_share(float x, float big, float T, unsigned long long total) {
  return __fdiv_rn(x == big ? 0.0f : x - big, T) - logf((float)total * 5.684341886e-14f);
}

struct Found {
  uint32_t key;                // the key (its leading bits) in which the count is reached
  float above, at;             // the count of larger keys, and of this one
};

// Masses are whole units. A share of one, rounded down, and whether that left a rest: what lies before a place is less than the
// share where it is less than `units`, or as much and there is a rest.
struct Share {
  unsigned long long units;
  bool rest;
  __device__ __forceinline__ Share(unsigned long long mass, float share) {
    const unsigned long long p64 = share > 0.0f ? __float2ull_rz(share * 18446744073709551616.0f) : 0ull;
    units = __umul64hi(mass, p64);
    rest = mass * p64 != 0;
  }
  __device__ __forceinline__ bool above(unsigned long long sum) const { return sum < units || (sum == units && rest); }
};

template <typename EI> constexpr int key_shift() {         // bits of the key that a logit of this type leaves alone
  return std::is_same<EI, BF16>::value ? 16 : std::is_same<EI, F16>::value ? 13 : 0;
}

// CUT: some row may have a top_k, top_p or min_p
template <typename EI, int E8, int NT, bool CUT>
__global__ void __launch_bounds__(NT, NT == 256 ? (E8 > 3 ? 2 : 4) : (E8 > 2 ? 1 : 2)) sample_kernel(Params p, int* __restrict__ err) {
  using TI = typename EI::T;
  constexpr int SH = key_shift<EI>(), BITS = 32 - SH;
  extern __shared__ __align__(16) uint8_t raw[];
  constexpr int WARPS = NT / 32;
  Smem<NT, CUT>& sm = *reinterpret_cast<Smem<NT, CUT>*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n_cta;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n_cta));
  const int rank = (int)cluster_ctarank();
  const long long row = blockIdx.x / n_cta;
  cluster_arrive();                                        // waited for before anything is written to another CTA
  Exchange exchange{sm, rank, n_cta, warp, lane};
  // the row's settings, checked by every thread alike
  const float u = p.u[row], T = p.temperature ? p.temperature[row] : 1.0f;
  const int top_k = CUT && p.top_k ? p.top_k[row] : 0;
  const float top_p = CUT && p.top_p ? p.top_p[row] : 1.0f, min_p = CUT && p.min_p ? p.min_p[row] : 0.0f;
  const bool first = rank == 0 && threadIdx.x == 0;
  if (!(u >= 0.0f && u < 1.0f) || !(T == 0.0f || (T >= T_MIN && T <= T_MAX)) || top_p != top_p || min_p != min_p) {
    cluster_wait();
    if (first) {
      p.tokens[row] = -1;
      if (p.logprob) p.logprob[row] = CUDART_NAN_F;
      report_device_error(err, DEVERR_INDEX);
    }
    return;                                                // the whole cluster
  }
  // ---- the row, eight values a vector; what lies outside it counts as -infinity
  const TI* x0 = reinterpret_cast<const TI*>(p.logits) + row * p.ld;
  const int off = p.vectors ? 0 : (int)((reinterpret_cast<uintptr_t>(x0) & 15) / sizeof(TI));
  const bool wide = !p.vectors || (reinterpret_cast<uintptr_t>(x0) & 15) == 0;
  const int nv = p.vectors ? p.vectors : (p.V + off + 7) / 8;
  const int v0 = (int)((long long)nv * rank / n_cta), v1 = (int)((long long)nv * (rank + 1) / n_cta);
  const int mine = v0 + warp * 32 * E8 + lane;             // vector i: mine + 32 i
  float x[E8][8];
#pragma unroll
  for (int i = 0; i < E8; ++i) {
    const int v = mine + 32 * i, at = 8 * v - off;
    if (v < v1 && wide && at >= 0 && at + 8 <= p.V) {
      unpack8<EI>(x0 + at, x[i]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[i][k] = v < v1 && at + k >= 0 && at + k < p.V ? (float)x0[at + k] : -CUDART_INF_F;
    }
  }
  for (int i = threadIdx.x; i < ROOTS; i += NT) sm.roots[i] = d_roots[i];
  uint32_t top = 0, own_top;
#pragma unroll
  for (int i = 0; i < E8; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[i][k] += 0.0f;                                     // -0 is 0
      top = max(top, key_of(x[i][k]));
    }
  own_top = top;
  top = __reduce_max_sync(0xffffffffu, top);
  if (threadIdx.x < 32) sm.part[threadIdx.x] = 0;
  __syncthreads();
  if (lane == 0) sm.part[warp] = top;
  __syncwarp();
  cluster_wait();                                          // every CTA of the cluster runs
  {
    const uint32_t (*all)[WIDE] = exchange();
    uint32_t m = 0;
    for (int r = 0; r < n_cta; ++r) m = max(m, all[r][lane]);
    top = __reduce_max_sync(0xffffffffu, m);
  }
  if (top == 0xFFFFFFFFu || top <= key_of(-CUDART_INF_F)) {            // a NaN, or nothing to draw from
    if (first) {
      p.tokens[row] = -1;
      if (p.logprob) p.logprob[row] = CUDART_NAN_F;
    }
    return;
  }
  const float big = of_key(top);
  if (T == 0.0f || top_k == 1) {
    // ---- the first of the largest
    uint32_t at = 0xFFFFFFFFu;
#pragma unroll
    for (int i = E8 - 1; i >= 0; --i)
#pragma unroll
      for (int k = 7; k >= 0; --k)
        if (x[i][k] == big) at = (uint32_t)(8 * (mine + 32 * i) - off + k);
    at = __reduce_min_sync(0xffffffffu, at);
    __syncthreads();
    if (threadIdx.x < 32) sm.part[threadIdx.x] = 0xFFFFFFFFu;
    __syncthreads();
    if (lane == 0) sm.part[warp] = at;
    const uint32_t (*all)[WIDE] = exchange();
    if (rank == 0 && warp == 0) {
      for (int r = 0; r < n_cta; ++r) at = min(at, all[r][lane]);
      at = __reduce_min_sync(0xffffffffu, at);
      if (lane == 0) {
        p.tokens[row] = (int)at;
        if (p.logprob) p.logprob[row] = 0.0f;
      }
    }
    return;
  }
  // log2(e) / T as two fp32 numbers
  const float ch = __fdiv_rn(1.44269502f, T), cl = __fdiv_rn(fmaf(-ch, T, 1.44269502f) + 1.92596299e-8f, T);

  const bool by_k = top_k > 0 && top_k < p.V, by_p = top_p < 1.0f;
  const unsigned long long floor_w = min_p > 0.0f ? (unsigned long long)(fminf(min_p, 1.0f) * 17592186044416.0f) : 0ull;

  // The next vector of the thread's comes first: code for one of them that goes around them all.
  auto around = [&]() {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float first_x = x[0][k];
#pragma unroll
      for (int i = 0; i + 1 < E8; ++i) x[i][k] = x[i + 1][k];
      x[E8 - 1][k] = first_x;
    }
  };
  uint32_t least = 0;                                      // kept: keys above it, and the first `ties` of those equal to it
  uint32_t ties = 0xFFFFFFFFu;
  if constexpr (CUT) {
  unsigned long long mass = 0, hist = 0;                   // of the row, and of this lane's part of it
  // A value's place: how far it lies below the largest, 2^32 steps of it down to where weights end; counted from the far end, so
  // that larger logits have larger places. Equal logits have the same one, and a few neighbours may.
  const float per = ch * (32.0f / 45.0f * 134217728.0f);
  auto place_of = [&](float v) -> uint32_t { return v == big ? 0xFFFFFFFFu : ~__float2uint_rz((big - v) * per); };
  // The CTA's mass of the values in each of 32 bins, into `part`. A weight is two words of 22 bits, so that the sums of two
  // threads' values are plain words, in any order.
  auto tally = [&](auto bin_of) {
    const int half = (int)threadIdx.x / (NT / 2), col = (int)threadIdx.x % (NT / 2);
    __syncthreads();
#pragma unroll
    for (int b = 0; b < 32; ++b) sm.halves[half][b][col] = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < E8; ++i, around())
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t bin = bin_of(x[0][k]);
        if (bin < 32u) {
          const unsigned long long w = weight(sm.roots, x[0][k], big, ch, cl);
          atomicAdd(&sm.halves[0][bin][col], (uint32_t)w & 0x3FFFFFu);
          atomicAdd(&sm.halves[1][bin][col], (uint32_t)(w >> 22));
        }
      }
    __syncthreads();
#pragma unroll
    for (int b = warp; b < 32; b += WARPS) {
      unsigned long long s = 0;
#pragma unroll
      for (int c = 0; c < NT / 2; c += 32) s += sm.halves[0][b][c + lane] + ((unsigned long long)sm.halves[1][b][c + lane] << 22);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) *reinterpret_cast<unsigned long long*>(&sm.part[MASSES + 2 * b]) = s;
    }
  };
  auto collect = [&](const uint32_t (*all)[WIDE]) -> unsigned long long {      // a bin a lane
    unsigned long long s = 0;
    for (int r = 0; r < n_cta; ++r) s += *reinterpret_cast<const unsigned long long*>(&all[r][MASSES + 2 * lane]);
    return s;
  };
  // the bin in which the goal is reached, with `above` in larger ones of an earlier pass; `sum`: over a lane's bin and the larger ones
  auto bin_of_goal = [&](const Share& goal, unsigned long long above, unsigned long long& sum) -> int {
    sum = hist;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long v = __shfl_down_sync(0xffffffffu, sum, o);
      if (lane + o < 32) sum += v;
    }
    return 31 - __clz(__ballot_sync(0xffffffffu, hist && !goal.above(above + sum)));
  };
  auto over_lanes = [](unsigned long long s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  };
  // ---- few kept: the `most` largest logits are sought, sorted and drawn from. Where the threads' own largest
  // are sorted, at least `most` values are not below the one at place `most`, and the CTA's `most` largest are
  // among them: a CTA lists all such values, and the first `most` of the sorted list of all CTAs are the row's.
  const int most = by_k ? (top_k <= NT ? top_k : 0) : (by_p || floor_w ? GUESS : 0);
  if (most) {
    auto& few = sm.few;
    uint32_t v = own_top;                                  // sorted by falling key, a value a thread
#pragma unroll
    for (int size = 2; size <= NT; size *= 2) {
#pragma unroll
      for (int stride = size / 2; stride > 0; stride /= 2) {
        uint32_t other;
        if (stride >= 32) {
          __syncthreads();
          few.keys[threadIdx.x] = v;
          __syncthreads();
          other = few.keys[threadIdx.x ^ stride];
        } else {
          other = __shfl_xor_sync(0xffffffffu, v, stride);
        }
        const bool larger = ((threadIdx.x & size) == 0) == ((threadIdx.x & stride) == 0);
        v = larger ? max(v, other) : min(v, other);
      }
    }
    __syncthreads();
    few.keys[threadIdx.x] = v;
    __syncthreads();
    const uint32_t least = max(few.keys[most - 1], key_of(-CUDART_INF_F) + 1u);
    uint32_t count = 0;
#pragma unroll
    for (int i = 0; i < E8; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) count += key_of(x[i][k]) >= least;
    uint32_t upto = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) sm.part[warp] = upto;
    const bool by_mass = by_p && !by_k;
    if (by_mass) {
      tally([&](float v) { return place_of(v) >> 27; });
      if (threadIdx.x == 0) sm.part[MASSES + 64] = place_of(of_key(least)) >> 27;
    }
    const uint32_t (*all)[WIDE] = exchange(by_mass);
    uint32_t n = 0, at = 0;                                // candidates, and those before this warp's
    for (int r = 0; r < n_cta; ++r) {
      const uint32_t c = lane < WARPS ? all[r][lane] : 0u;
      n += c;
      if (r < rank || (r == rank && lane < warp)) at += c;
    }
    n = __reduce_add_sync(0xffffffffu, n);
    at = __reduce_add_sync(0xffffffffu, at) + upto - count;
    bool listed = n <= LIST;
    if (by_mass) {
      hist = collect(all);
      mass = over_lanes(hist);
      // the border lies below every CTA's listed ones, and with it below the `most` largest: what would be listed is not enough
      uint32_t bin = 0;
      for (int r = 0; r < n_cta; ++r) bin = max(bin, all[r][MASSES + 64]);
      unsigned long long sum;
      listed = listed && (floor_w || bin_of_goal(Share(mass, top_p), 0ull, sum) >= (int)bin);
    }
    if (listed) {
      uint32_t list;                                       // the first CTA's
      asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(list) : "r"(smem_u32(few.list)));
      if (count) {
#pragma unroll
        for (int i = 0; i < E8; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t key = key_of(x[i][k]);
            if (key >= least) {
              const uint32_t idx = (uint32_t)(8 * (mine + 32 * i) - off + k);
              asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(list + 8 * at), "l"((unsigned long long)key << 32 | (0xFFFFFFFFu - idx))
                           : "memory");
              ++at;
            }
          }
      }
      __syncwarp();
      cluster_sync();
      bool done = by_k;
      if (rank == 0) {
        int size2 = 2;
        while (size2 < (int)n) size2 *= 2;
        for (int i = (int)n + threadIdx.x; i < size2; i += NT) few.list[i] = 0;
        for (int size = 2; size <= size2; size *= 2)
          for (int stride = size / 2; stride > 0; stride /= 2) {
            __syncthreads();
            for (int i = threadIdx.x; i < size2 / 2; i += NT) {
              const int lo = 2 * i - (i & (stride - 1)), hi = lo + stride;
              const unsigned long long a = few.list[lo], b = few.list[hi];
              if ((a < b) == ((lo & size) == 0)) {
                few.list[lo] = b;
                few.list[hi] = a;
              }
            }
          }
        __syncthreads();
        const int m = min(most, (int)n), i = threadIdx.x;
        const unsigned long long mine_e = i < m ? few.list[i] : 0ull;
        const float xi = of_key((uint32_t)(mine_e >> 32));
        unsigned long long w = i < m ? weight(sm.roots, xi, big, ch, cl) : 0ull, sum = w;
        // sums up to here, over all threads
        auto scan = [&](unsigned long long& s, unsigned long long& total) {
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
          }
          __syncthreads();
          if (lane == 31) few.sums[warp] = s;
          __syncthreads();
          total = 0;
          unsigned long long before = 0;
          for (int k = 0; k < WARPS; ++k) {
            const unsigned long long y = few.sums[k];
            total += y;
            if (k < warp) before += y;
          }
          s += before;
        };
        unsigned long long total;
        scan(sum, total);
        const Share goal(by_k ? total : mass, by_p ? top_p : 0.0f);
        const bool keep = i < m && w >= floor_w && (i == 0 || !by_p || goal.above(sum - w));
        // whether what may be kept lies among the sorted ones, where their number was a guess
        done = by_k || (int)n < most || (by_p && !goal.above(total)) || (floor_w && __syncthreads_or(i == m - 1 && w < floor_w));
        if (!keep) w = 0;
        if (done) {
          const int kept = __syncthreads_count(keep);      // the first ones
          few.w[i] = w;
          sum = w;
          scan(sum, total);
          const unsigned long long target = __umul64hi(total, __float2ull_rz(u * 18446744073709551616.0f));
          if (keep) {
            // the kept ones before it by index: those whose lower word is larger
            const uint32_t low = (uint32_t)mine_e;
            unsigned long long less = 0;
            for (int j = 0; j < kept; ++j)
              if ((uint32_t)few.list[j] > low) less += few.w[j];
            if (target >= less && target - less < w) {
              p.tokens[row] = (int)(0xFFFFFFFFu - low);
              if (p.logprob) p.logprob[row] = log_share(xi, big, T, total);
            }
          }
        }
      }
      if (by_k) return;
      if (threadIdx.x < 32) sm.part[threadIdx.x] = done;
      if (exchange()[0][0]) return;
      __syncthreads();
    }
  }

  // ---- where the count of values, by falling logit, reaches `target`
  auto find = [&](float target) -> Found {
    uint32_t prefix = 0;
    float above = 0.0f, at = 0.0f;
#pragma unroll 1
    for (int left = BITS; left > 0;) {
      const int nb = min(5, left);
      left -= nb;
#pragma unroll
      for (int b = 0; b < 32; ++b) sm.bins[b][threadIdx.x] = 0.0f;
#pragma unroll
      for (int i = 0; i < E8; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t bin = (key_of(x[i][k]) >> SH >> left) - (prefix << nb);
          if (bin < (1u << nb)) sm.bins[bin][threadIdx.x] += 1.0f;
        }
      __syncthreads();
#pragma unroll
      for (int b = warp; b < 32; b += WARPS) {
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < NT; c += 32) s += sm.bins[b][c + lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) sm.part[b] = __float_as_uint(s);
      }
      const uint32_t (*all)[WIDE] = exchange();
      float own = 0.0f;
      for (int r = 0; r < n_cta; ++r) own += __uint_as_float(all[r][lane]);
      float sum = own;                                     // over this bin and the larger ones
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float v = __shfl_down_sync(0xffffffffu, sum, o);
        if (lane + o < 32) sum += v;
      }
      const int b = 31 - __clz(__ballot_sync(0xffffffffu, own > 0.0f && above + sum >= target));
      const float over = __shfl_sync(0xffffffffu, sum, min(b + 1, 31));
      above += b < 31 ? over : 0.0f;
      at = __shfl_sync(0xffffffffu, own, b);
      prefix = (prefix << nb) + (uint32_t)b;
    }
    return Found{prefix, above, at};
  };
  unsigned long long beyond = 0;                           // the mass of equal ones that top_k leaves out
  if (by_k) {
    const Found f = find((float)top_k);
    least = f.key;
    ties = (uint32_t)max(1, top_k - (int)f.above);
    if ((float)ties >= f.at) ties = 0xFFFFFFFFu;
    else beyond = weight(sm.roots, of_lead<SH>(least), big, ch, cl) * ((uint32_t)f.at - ties);
  }
  if (by_p) {
    // ---- the border's key: the bits of its place are fixed five at a time, until few values are left, then those of the key
    constexpr int LEVELS = SH ? 2 : 4;
    uint32_t prefix = 0, place = 0;                        // leading bits of the key, at first of the place; the place's, once fixed
    int left = 32, place_left = 0, nb = 5;
    bool keys = false, have = !by_k;
    unsigned long long above = 0;                          // the mass of larger ones
    Share goal(mass, top_p);
#pragma unroll 1
    for (;;) {
      left -= nb;
      if (!have) {
        tally([&](float v) -> uint32_t {
          const uint32_t k = key_of(v) >> SH, at = place_of(v);
          const bool in = k >= least && (!keys || at >> place_left == place);
          const uint32_t bin = ((keys ? k : at) >> left) - (prefix << nb);
          return in && bin < (1u << nb) ? bin : 32u;
        });
        hist = collect(exchange(true));
        if (by_k && !keys && left == 27) goal = Share(mass = over_lanes(hist) - beyond, top_p);
      }
      have = false;
      unsigned long long sum;
      const int b = bin_of_goal(goal, above, sum);
      const unsigned long long over = __shfl_sync(0xffffffffu, sum, min(b + 1, 31));
      above += b < 31 ? over : 0ull;
      prefix = (prefix << nb) + (uint32_t)b;
      if (!keys && left > 32 - 5 * LEVELS) continue;
      if (!keys) {
        // the keys that are left
        place = prefix;
        place_left = left;
        uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll 1
        for (int i = 0; i < E8; ++i, around())
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t v = key_of(x[0][k]) >> SH;
            if (v >= least && place_of(x[0][k]) >> left == place) {
              lo = min(lo, v);
              hi = max(hi, v);
            }
          }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
          sm.part[warp] = hi;
          sm.part[WARPS + warp] = ~lo;
        }
        const uint32_t (*all)[WIDE] = exchange();
        uint32_t most_of = 0;                              // the upper half of the lanes: inverted smallest
        for (int r = 0; r < n_cta; ++r) most_of = max(most_of, all[r][lane]);
        hi = __reduce_max_sync(0xffffffffu, lane < WARPS ? most_of : 0u);
        lo = ~__reduce_max_sync(0xffffffffu, lane < WARPS ? 0u : most_of);
        keys = true;
        left = lo == hi ? 0 : 32 - __clz(lo ^ hi);
        prefix = left < 32 ? hi >> left : 0u;
      }
      if (left == 0) break;
      nb = min(5, left);
    }
    const uint32_t key = prefix;
    // of the equal ones as many as begin below the goal
    const unsigned long long w = weight(sm.roots, of_lead<SH>(key), big, ch, cl), gap = goal.units - above, whole = gap / w;
    const uint32_t n = (uint32_t)max(1ull, whole + (goal.rest || whole * w < gap));
    ties = key == least ? min(ties, n) : n;
    least = key;
  }
  }
  // ---- how many values equal to the border lie before this warp's
  uint32_t before = 0;
  const bool cut = ties != 0xFFFFFFFFu;
  if (cut) {
    uint32_t eq = 0;
#pragma unroll
    for (int i = 0; i < E8; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) eq += key_of(x[i][k]) >> SH == least;
    eq = __reduce_add_sync(0xffffffffu, eq);
    __syncthreads();
    if (threadIdx.x < 32) sm.part[threadIdx.x] = 0;
    __syncthreads();
    if (lane == 0) sm.part[warp] = eq;
    const uint32_t (*all)[WIDE] = exchange();
    for (int r = 0; r <= rank; ++r)
      if (r < rank || lane < warp) before += all[r][lane];
    before = __reduce_add_sync(0xffffffffu, before);
  }

  // ---- the weights of a vector's kept values in units of 2^-44; `eq` counts the warp's equal ones so far
  auto weights = [&](const float (&xi)[8], uint32_t& eq, unsigned long long (&w)[8]) {
    uint32_t at = 0;
    if (cut) {
      uint32_t n = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) n += key_of(xi[k]) >> SH == least;
      uint32_t upto = n;
      if (__any_sync(0xffffffffu, n != 0)) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
      }
      at = eq + upto - n;
      eq += __shfl_sync(0xffffffffu, upto, 31);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t key = key_of(xi[k]) >> SH;
      bool keep = key > least;
      if (key == least) {
        keep = !cut || at < ties;
        ++at;
      }
      w[k] = 0;
      if (keep) {
        w[k] = weight(sm.roots, xi[k], big, ch, cl);
        if (CUT && w[k] < floor_w) w[k] = 0;
      }
    }
  };
  // f on every vector in turn: they go around and the first is worked on. Unrolled, the code of all weights would be read
  // from memory, once (256 rows of 151665, in us, so / unrolled: whole 177 / 264, with top_p alone 894 / 934).
  auto in_turn = [&](auto&& f) {
#pragma unroll 1
    for (int i = 0; i < E8; ++i, around()) f(i, x[0]);
  };
  unsigned long long own = 0;
  uint32_t eq = before;
  in_turn([&](int, const float (&xi)[8]) {
    unsigned long long w[8];
    weights(xi, eq, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) own += w[k];
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);
  __syncthreads();
  if (lane == 0) {
    sm.part[2 * warp] = (uint32_t)own;
    sm.part[2 * warp + 1] = (uint32_t)(own >> 32);
  }
  const uint32_t (*all)[WIDE] = exchange();
  unsigned long long total = 0, less = 0;                  // the kept mass, and what lies before this warp
  if (lane < WARPS) {
    for (int r = 0; r < n_cta; ++r) {
      const unsigned long long v = *reinterpret_cast<const unsigned long long*>(&all[r][2 * lane]);
      total += v;
      if (r < rank || (r == rank && lane < warp)) less += v;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    less += __shfl_xor_sync(0xffffffffu, less, o);
  }
  const unsigned long long target = __umul64hi(total, __float2ull_rz(u * 18446744073709551616.0f));
  if (target < less || target - less >= own) return;
  // ---- this warp has the token
  eq = before;
  in_turn([&](int i, const float (&xi)[8]) {
    unsigned long long w[8], sum = 0;
    weights(xi, eq, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += w[k];
    unsigned long long upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    unsigned long long at = less + upto - sum;
    if (target >= at && target - at < sum) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (target >= at && target - at < w[k]) {
          p.tokens[row] = 8 * (mine + 32 * i) - off + k;
          if (p.logprob) p.logprob[row] = log_share(xi[k], big, T, total);
        }
        at += w[k];
      }
    }
    less += __shfl_sync(0xffffffffu, upto, 31);
  });
}

template <typename EI, int E8, int NT, bool CUT>
gptq_status launch(const Params& p, long long rows, int c, cudaStream_t s) {
  static PerDevice done;
  if (gptq_status st = allow_smem(done, sample_kernel<EI, E8, NT, CUT>, sizeof(Smem<NT, CUT>), "sample_kernel")) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * c));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = sizeof(Smem<NT, CUT>);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, sample_kernel<EI, E8, NT, CUT>, p, device_error_word());
  count_launch();
  return check_launch("sample_kernel");
}

template <typename EI>
gptq_status pick(Params p, long long rows, cudaStream_t s) {
  const int sms = sm_count();
  const bool cut = p.top_k || p.top_p || p.min_p;
  // vectors of a row, were it to begin in the middle of 16 bytes
  int nv = (p.V + 14) / 8;
  if (nv > MOST * 512 * 8) {
    nv = (p.V + 7) / 8;
    p.vectors = nv;
  }
  // Whole rows: blocks of 256 threads, more of which share an SM and work while others wait for their cluster.
  // Cut rows: of 512, whose largest values are sorted, and few of them, as each lists its own.
  const int nt = cut || nv > MOST * 256 * 10 ? 512 : 256, fit = cut ? CUTS : nt == 512 ? 8 : WHOLE;
  int c = 1;
  while (c < MOST && (nv > (long long)c * nt * fit || (rows * c <= sms && nv > c * 256))) c *= 2;
  const int e = (nv + c * nt - 1) / (c * nt);
  auto go = [&](auto e8) -> gptq_status {
    constexpr int E8 = decltype(e8)::value;
    if (cut) return launch<EI, E8, 512, true>(p, rows, c, s);
    if constexpr (E8 == 8)
      if (nt == 512) return launch<EI, 8, 512, false>(p, rows, c, s);
    return launch<EI, E8, 256, false>(p, rows, c, s);
  };
  if (!cut && nt == 512) return go(std::integral_constant<int, 8>{});
  switch (e) {
    case 1: return go(std::integral_constant<int, 1>{});
    case 2: return go(std::integral_constant<int, 2>{});
    case 3:
    case 4: return go(std::integral_constant<int, 4>{});
    case 5: return go(std::integral_constant<int, 5>{});
    case 6:
    case 7:
    case 8: return go(std::integral_constant<int, 8>{});
    default: return launch<EI, 10, 256, false>(p, rows, c, s);
  }
}

}  // namespace smp
}  // namespace gptq
