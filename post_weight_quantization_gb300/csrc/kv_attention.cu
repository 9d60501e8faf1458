// Attention of a few query tokens per sequence over the 4-bit paged cache (decoding).
//
//   o_i = sum_j p_ij v_j,   p_i = softmax over the seen j of sm_scale * q_i . k_j
//   k_j = kc_j ks_j + kl_j (codes, scale, lowest value; v_j alike), so
//   q_i . k_j = ks_j (q_i . kc_j) + kl_j sum(q_i),    o_i = sum_j (p_ij vs_j) vc_j + sum_j p_ij vl_j
//
// One pass over the cache with a running maximum and sum; both products run on the tensor
// cores with the codes themselves as an operand, taken from the packed words in registers:
//   * A pair of codes masked out of a word (0x000F000F) IS a pair of fp16 numbers, code *
//     2^-24 (subnormal), and 0x00F000F0 is the pair code * 2^-20: no conversion, two
//     logic instructions per four codes. The powers of two leave with the scale (K: into
//     the query; V: at the end). Products with the fp16 query are exact in fp32.
//   * Each query row is scaled by the power of two that brings its largest value to
//     [2^14, 2^15), so a bf16 query is exact in fp16 too.
//   * S^T = K Q^T: A = 16 keys x 16 dims of codes, B = the query rows (N = 8). The fp32
//     scores leave with their key on the lane row; one movmatrix per 8 x 8 tile brings
//     the probabilities to the B layout of O^T = V^T P^T (A = 16 dims x 16 keys of codes).
//   * The probabilities times the key's V scale are rounded to fp16 for the second product:
//     2^-11 of each, random in sign, against the output's own 2^-8 for bf16. For fp16 outputs, which
//     round to 2^-11 themselves, they are two fp16 parts (22 bits) and two products: with one, the
//     error against 64 bits was 1.1 to 1.56 times the output's rounding, with two it is 1.00 (and two
//     sequences of 131000 keys take 74 instead of 69 us, 48 ragged ones 45 instead of 43). They are
//     brought to the top of fp16's range by a power of two that follows the largest V scale
//     seen, so small probabilities keep their bits down to 2^-24 of the largest.
//   Why mma.sync and not tcgen05: the product is bound by HBM bandwidth (one pass over the
//   cache for at most 16 or 32 rows), and tcgen05 would need the codes unpacked to 16 bits in
//   shared memory, four times the bytes that come from HBM, where here they go from the
//   packed words to the tensor core through registers.
//
// Work: a sequence's (kv head, 8 NT query rows) is an item of tiles of 128 keys; the tiles of
// all items form one line that is cut into equal pieces, one per CTA, from the lengths on the
// device. Tiles arrive in a ring of bulk copies (whole pages where a page is 16 ... 128 keys, a
// power of two), which the CTA's four warps issue in turn. Each warp takes 32 keys of every
// tile with its own running maximum; they meet at the item's end. An item
// that is cut between CTAs leaves unnormalised parts in the workspace, which
// kv_join_kernel joins in a fixed order.
//
// Bound: HBM bandwidth. Measured, 64 + 8 heads of 128: two sequences of 120000 and 131001 keys 69 us (273
// MB, 3.9 TB/s with the join, 6 TB/s in the loop), 48 of 60 to 4099 keys 43 us; the start (lengths, page
// table, first copies) and the join's launch take about 10 us of each.
#include "kv_line.cuh"

namespace gptq {
namespace kva {

constexpr int WARPS = 4, THREADS = WARPS * 32;
constexpr int KC = TILE / WARPS;                // keys of a warp's chunk
constexpr int kItemCost = 2;                    // what beginning an item costs, in tiles
constexpr float kSlack = 6.0f;                  // a row's maximum may lag by 2^6 before it is moved
constexpr int kVExp = 8;                        // V scales are brought below 2^(kVExp + 1)

template <int D, int NT>
struct Cfg {
  static constexpr int R = 8 * NT;
  static constexpr int STAGE = TILE * (D + 8);  // K codes, V codes, numbers of a tile
  static constexpr int NS = D == 256 ? 2 : 3;
  static constexpr int RED_LD = D + 4;
  static constexpr int RED = WARPS * 8 * RED_LD * 4;
  static constexpr int RING = NS * STAGE;
  static constexpr int BIG = RING + RED;
  static constexpr int SMEM = BIG + 112 + 2 * NS * 8 + 3 * WARPS * R * 4;
  static constexpr int OCC = D == 256 || NT == 4 ? 2 : NT == 2 ? (D == 64 ? 3 : 2) : (D == 64 ? 4 : 3);
  static constexpr int PART = R * D + 2 * R;    // floats of one part
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(addr + 4 * i));
  }
}

// A warp's running state over an item's keys. In the scores' C layout a lane (g = lane / 4,
// t = lane % 4) holds keys g and g + 8 of a 16-key tile for rows 2t and 2t + 1 of each n-tile;
// in the output's, dims of its V words for the same two rows.
template <int D, int NT>
struct State {
  float o[D / 16][NT][4];
  float mrc[NT][2];              // running maximum in log2 units (0 while there is none)
  float thr[NT][2];              // mrc + kSlack (-inf while there is none)
  float l[NT][2], low[NT][2];    // this lane's part of sum p and sum p * vl
  uint32_t q[NT][D / 8];         // B fragments: 4 registers per word of the lane's K words
  float rowc[NT][2], rq[NT][2];  // log2 units per inner score; the scaled query's sum
  int lo[NT][2], hi[NT][2];      // the keys the row sees: lo ... hi
  float vlim, vinv;              // V scales below vlim = 2^(x+1) are multiplied by vinv = 2^(kVExp - x)
};

template <int D, int NT, bool FINE, bool MASK>
__device__ __forceinline__ void chunk(State<D, NT>& st, uint32_t k_0, uint32_t k_1, uint32_t n_0, uint32_t n_1, uint32_t pb,
                                      int key0, int g, int t) {
  constexpr int KW = D / 32;                     // K words of a key per lane, words KW t ...
  constexpr int VW = D / 64;                     // V words of a key per lane, words VW g ...
  constexpr int RB = D / 2;                      // bytes of a row of codes
  // the chunk's two 16-key tiles start at k_0 and k_1; a block of pb keys holds K codes, V codes, numbers
  const int sw = (g >> 1) & 1;                   // tile row r holds key r ^ ((r >> 1) & 1): fewer bank conflicts in V
  const int kr = g ^ sw;

  float s[2][NT][4];
  float vs[2][2], vl[2][2];
  {
    // four independent accumulation chains: the two 16-key tiles, two MMAs of each word
    uint32_t wa[2][KW], wb[2][KW];
    float s2[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t kb = (mt ? k_1 : k_0) + kr * RB + t * KW * 4;
      lds_words<KW>(kb, wa[mt]);
      lds_words<KW>(kb + 8 * RB, wb[mt]);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[mt][n][i] = s2[mt][n][i] = 0.0f;
    }
#pragma unroll
    for (int w = 0; w < KW; ++w)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint32_t a = wa[mt][w], c = wb[mt][w], a8 = a >> 8, c8 = c >> 8;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(s[mt][n], a & 0x000F000Fu, c & 0x000F000Fu, a & 0x00F000F0u, c & 0x00F000F0u, st.q[n][4 * w],
                  st.q[n][4 * w + 1]);
          mma_f16(s2[mt][n], a8 & 0x000F000Fu, c8 & 0x000F000Fu, a8 & 0x00F000F0u, c8 & 0x00F000F0u,
                  st.q[n][4 * w + 2], st.q[n][4 * w + 3]);
        }
      }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[mt][n][i] += s2[mt][n][i];
  }
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    // numbers of the lane's two keys; inner = ks 2^24 acc + kl sum(q)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t num[2];
      const int r = 16 * mt + kr + 8 * e;
      lds_words<2>((mt ? n_1 : n_0) + (kr + 8 * e) * 8, num);
      float2 kn = __half22float2(*reinterpret_cast<const __half2*>(&num[0]));
      float2 vn = __half22float2(*reinterpret_cast<const __half2*>(&num[1]));
      const float ks = kn.x * 16777216.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = fmaf(kn.y, st.rq[n][i], s[mt][n][2 * e + i] * ks);
          if (MASK && (key0 + r > st.hi[n][i] || key0 + r < st.lo[n][i])) x = -CUDART_INF_F;
          s[mt][n][2 * e + i] = x;
        }
      vs[mt][e] = vn.x;
      vl[mt][e] = vn.y;
    }
  }
  // V scales above the range in use move it (a power of two: exact)
  {
    float vm = fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1]));
    if (MASK) {                                  // places past the keys may hold anything: rows decide
      vm = 0.0f;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          bool any = false;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) any |= s[mt][n][2 * e + i] != -CUDART_INF_F;
          if (any) vm = fmaxf(vm, vs[mt][e]);
        }
    }
    if (__any_sync(0xffffffffu, vm >= st.vlim)) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
      const int x = (int)(__float_as_uint(vm) >> 23) - 127;          // a finite fp16 value: -24 ... 15
      const float vinv = pow2(kVExp - x), f = vinv / st.vinv;
      st.vinv = vinv;
      st.vlim = pow2(x + 1);
#pragma unroll
      for (int m = 0; m < D / 16; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) st.o[m][n][i] *= f;
    }
  }
  // running maximum, moved only when a score passes it by 2^kSlack
  {
    float mx[NT][2];
    bool over = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[n][i] = fmaxf(fmaxf(s[0][n][i], s[0][n][2 + i]), fmaxf(s[1][n][i], s[1][n][2 + i])) * st.rowc[n][i];
        over |= mx[n][i] > st.thr[n][i];
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v = mx[n][i];
#pragma unroll
          for (int o = 4; o <= 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
          const bool had = st.thr[n][i] != -CUDART_INF_F;
          v = had ? fmaxf(v, st.mrc[n][i]) : v;
          if (v != -CUDART_INF_F) {
            const float f = had ? ex2(st.mrc[n][i] - v) : 0.0f;
            st.mrc[n][i] = v;
            st.thr[n][i] = v + kSlack;
            st.l[n][i] *= f;
            st.low[n][i] *= f;
#pragma unroll
            for (int m = 0; m < D / 16; ++m) {
              st.o[m][n][i] *= f;
              st.o[m][n][2 + i] *= f;
            }
          }
        }
    }
  }
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    uint32_t b[NT][2], b2[NT][2];                // FINE: what the rounding left over
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float c = vs[mt][e] * st.vinv;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float pc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = s[mt][n][2 * e + i];
          const float pr = ex2(fmaf(x, st.rowc[n][i], -st.mrc[n][i]));
          if (MASK && x == -CUDART_INF_F) {      // unseen: its numbers may be anything
            pc[i] = 0.0f;
          } else {
            st.l[n][i] += pr;
            st.low[n][i] = fmaf(pr, vl[mt][e], st.low[n][i]);
            pc[i] = pr * c;
          }
        }
        const uint32_t h = pack_half2(pc[0], pc[1]);
        b[n][e] = movmatrix(h);
        if (FINE) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          b2[n][e] = movmatrix(pack_half2(pc[0] - f.x, pc[1] - f.y));
        }
      }
    }
    // V^T fragments: keys of tile rows 2t, 2t + 1 (low) and 2t + 8, 2t + 9 (high)
    const uint32_t vb = (mt ? k_1 : k_0) + pb * RB + g * VW * 4;
    const int r0 = (2 * t) ^ (t & 1), r1 = (2 * t + 1) ^ (t & 1);
    uint32_t v0[VW], v1[VW], v2[VW], v3[VW];
    lds_words<VW>(vb + r0 * RB, v0);
    lds_words<VW>(vb + r1 * RB, v1);
    lds_words<VW>(vb + (r0 + 8) * RB, v2);
    lds_words<VW>(vb + (r1 + 8) * RB, v3);
#pragma unroll
    for (int w = 0; w < VW; ++w)
#pragma unroll
      for (int by = 0; by < 4; ++by) {
        // byte `by` of the first key's word in the low half, of the second's in the high half
        const uint32_t sel = (uint32_t)(by * 0x0011 + (4 + by) * 0x1100);
        const uint32_t l2 = prmt(v0[w], v1[w], sel), h2 = prmt(v2[w], v3[w], sel);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(st.o[4 * w + by][n], l2 & 0x000F000Fu, l2 & 0x00F000F0u, h2 & 0x000F000Fu, h2 & 0x00F000F0u, b[n][0],
                  b[n][1]);
          if (FINE)
            mma_f16(st.o[4 * w + by][n], l2 & 0x000F000Fu, l2 & 0x00F000F0u, h2 & 0x000F000Fu, h2 & 0x00F000F0u, b2[n][0],
                    b2[n][1]);
        }
      }
  }
}



template <int D, int NT, bool FINE>
__global__ void __launch_bounds__(THREADS, Cfg<D, NT>::OCC) kv_split_kernel(Params p, int* __restrict__ err) {
  using C = Cfg<D, NT>;
  constexpr int R = C::R, NS = C::NS, KW = D / 32, VW = D / 64;
  extern __shared__ __align__(128) uint8_t smem[];
  float* join = reinterpret_cast<float*>(smem + C::RING);                                // [WARPS][8][RED_LD]: an n-tile at a time
  long long* sh = reinterpret_cast<long long*>(smem + C::BIG);                           // 14 values
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BIG + 112);
  uint64_t* empty = full + NS;
  float* red = reinterpret_cast<float*>(smem + C::BIG + 112 + 2 * NS * 8);               // maximum, sum, low sum: [3][WARPS][R]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem);
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], WARPS);
    }
    fence_mbar_init();
  }
  Line<R, kItemCost> line;
  line.init(p, sh, err);
  grid_dep_launch();
  // where this warp's two 16-key tiles lie in a stage: codes and numbers
  uint32_t koff[2], noff[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int k = warp * KC + 16 * m, blk = k >> p.pb_log2, at = k & (p.pb - 1);
    koff[m] = blk * p.pb * (D + 8) + at * (D / 2);
    noff[m] = blk * p.pb * (D + 8) + p.pb * D + at * 8;
  }

  // Lanes issue a tile's copies in the warp whose turn it is (tile i of the item is warp i % WARPS's).
  Copies cp;
  cp.init(p, lane);
  bool dead = false;
  auto issue = [&](uint32_t u, long long src) {
    const uint32_t st = u % NS;
    if (!mbar_wait_poll(&empty[st], (u / NS & 1u) ^ 1u, nullptr)) {
      if (lane == 0) report_device_error(err, DEVERR_TIMEOUT);
      dead = true;
      return;
    }
    cp.issue(p, ring + st * C::STAGE, &full[st], src, D, lane);
  };

  uint32_t slot = 0, phase = 0;                  // the ring's next tile
  uint32_t use = 0;                              // tiles taken from the ring so far, through all items
  Item it;
  bool have = line.next(p, it);
  int4 cut = make_int4(0, 0, 0, 0);
  if (have && warp < NS - 1 && warp < it.nt) issue(use + warp, cp.source(p, it, warp, D, err));

  while (have) {
    // this warp's next tile to issue, NS - 1 tiles before it is taken
    int ni = warp < NS - 1 ? warp + WARPS : warp;
    long long nsrc = cp.source(p, it, ni, D, err);
    const int pos0 = it.sq.len - it.sq.nq;

    // ---- the query rows as B fragments
    State<D, NT> st;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = it.rt * R + 8 * n + g;
      float mx = 0.0f, sum = 0.0f;
      uint4 raw[KW];
#pragma unroll
      for (int w = 0; w < KW; ++w) raw[w] = make_uint4(0u, 0u, 0u, 0u);
      if (8 * n + g < it.rows) {
        const int i = r / p.G, hq = it.h * p.G + r - i * p.G;
        const uint16_t* qp = reinterpret_cast<const uint16_t*>(p.Q) + (it.sq.tok0 + i) * p.ldq + (long long)hq * D + t * KW * 8;
#pragma unroll
        for (int w = 0; w < KW; ++w) raw[w] = *reinterpret_cast<const uint4*>(qp + 8 * w);
      }
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        float v[8];
        if (p.q_f16) unpack8<F16>(&raw[w], v); else unpack8<BF16>(&raw[w], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          mx = fmaxf(mx, fabsf(v[k]));
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = row_exponent(mx);
      const float f = pow2(e);
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        float v[8];
        if (p.q_f16) unpack8<F16>(&raw[w], v); else unpack8<BF16>(&raw[w], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[k] *= f;
          sum += v[k];                           // of the scaled values: the raw ones' sum can pass fp32
        }
        st.q[n][4 * w] = pack_half2(v[0], v[4]);
        st.q[n][4 * w + 1] = pack_half2(v[1] * 0.0625f, v[5] * 0.0625f);
        st.q[n][4 * w + 2] = pack_half2(v[2], v[6]);
        st.q[n][4 * w + 3] = pack_half2(v[3] * 0.0625f, v[7] * 0.0625f);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const float rs = sum, rc = p.scale_log2 * pow2(-e);
#pragma unroll
      for (int i = 0; i < 2; ++i) {              // rows 2t, 2t + 1 of the n-tile, from the lanes that read them
        st.rq[n][i] = __shfl_sync(0xffffffffu, rs, 4 * (2 * t + i));
        st.rowc[n][i] = __shfl_sync(0xffffffffu, rc, 4 * (2 * t + i));
        const int rr = 8 * n + 2 * t + i, tk = (it.rt * R + rr) / p.G;
        const long long lo = p.window > 0 ? (long long)pos0 + tk - p.window + 1 : 0;
        st.lo[n][i] = lo > 0 ? (lo < 0x7FFFFFFF ? (int)lo : 0x7FFFFFFF) : 0;
        st.hi[n][i] = rr >= it.rows ? -1 : (p.causal ? min(it.sq.len - 1, pos0 + tk) : it.sq.len - 1);
        st.mrc[n][i] = 0.0f;
        st.thr[n][i] = -CUDART_INF_F;
        st.l[n][i] = 0.0f;
        st.low[n][i] = 0.0f;
      }
#pragma unroll
      for (int m = 0; m < D / 16; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.o[m][n][i] = 0.0f;
    }
    st.vlim = pow2(-24);
    st.vinv = pow2(kVExp + 25);

    // ---- the tiles; this warp takes the keys 32 warp ... 32 warp + 31 of each. Tiles plain_lo
    // ... plain_hi need no mask: every row sees all their keys
    const int hi_min = p.causal ? min(it.sq.len, max(0, pos0 + it.i0 + 1)) : it.sq.len;
    const long long klo1 = p.window > 0 ? (long long)pos0 + it.i1 - p.window + 1 : 0;
    const int lo_max = klo1 > 0 ? (int)(klo1 < it.sq.len ? klo1 : it.sq.len) : 0;
    const int plain_lo = lo_max > warp * KC ? (lo_max - warp * KC + TILE - 1) / TILE - it.tl : -it.tl;
    const int plain_hi = (hi_min >= warp * KC + KC ? (hi_min - warp * KC - KC) / TILE : -1) - it.tl;
    for (int i = 0; i < it.nt && !dead; ++i) {
      if (i + NS - 1 == ni && ni < it.nt) {
        issue(use + NS - 1, nsrc);
        ni += WARPS;
        nsrc = cp.source(p, it, ni, D, err);
      }
      if (!mbar_wait_bounded(&full[slot], phase, nullptr)) {
        if (lane == 0) report_device_error(err, DEVERR_TIMEOUT);
        dead = true;
      }
      const uint32_t base = ring + slot * C::STAGE;
      const int key0 = (it.tl + i) * TILE + warp * KC;
      if (i >= plain_lo && i <= plain_hi)
        chunk<D, NT, FINE, false>(st, base + koff[0], base + koff[1], base + noff[0], base + noff[1], p.pb, key0, g, t);
      else if (key0 < it.hi_all && key0 + KC > it.lo_all)
        chunk<D, NT, FINE, true>(st, base + koff[0], base + koff[1], base + noff[0], base + noff[1], p.pb, key0, g, t);
      // the stage's words have been read: without the fence nothing keeps the next copy, which is
      // another proxy's write, behind loads that are still on their way to the MMAs
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      ++use;
      if (++slot == NS) {
        slot = 0;
        phase ^= 1u;
      }
    }

    // ---- the next item's first tiles are on their way while the warps meet over this one
    Item nx;
    const bool more = line.next(p, nx);
    if (more && !dead && warp < NS - 1 && warp < nx.nt) issue(use + warp, cp.source(p, nx, warp, D, err));

#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) {
          st.l[n][i] += __shfl_xor_sync(0xffffffffu, st.l[n][i], o);
          st.low[n][i] += __shfl_xor_sync(0xffffffffu, st.low[n][i], o);
        }
        if (g == 0) {
          const int r = 8 * n + 2 * t + i;
          red[warp * R + r] = st.thr[n][i] == -CUDART_INF_F ? (st.l[n][i] != 0.0f ? 0.0f : -CUDART_INF_F) : st.mrc[n][i];
          red[(WARPS + warp) * R + r] = st.l[n][i];
          red[(2 * WARPS + warp) * R + r] = st.low[n][i];
        }
      }
    float* ob = join + warp * 8 * C::RED_LD;
    const float ue = 16777216.0f / st.vinv, uo = ue * 0.0625f;
    float* out = p.part + (2LL * blockIdx.x + (it.lead ? 0 : 1)) * C::PART;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n) __syncthreads();                    // the n-tile before has been read
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
          for (int by = 0; by < 4; by += 2) {
            const int m = 4 * w + by;
            *reinterpret_cast<float4*>(ob + (2 * t + i) * C::RED_LD + (VW * g + w) * 8 + 2 * by) =
                make_float4(st.o[m][n][i] * ue, st.o[m][n][2 + i] * uo, st.o[m + 1][n][i] * ue, st.o[m + 1][n][2 + i] * uo);
          }
      dead = __syncthreads_or(dead);
      for (int x = tid; x < 8 * (D / 4); x += THREADS) {
        const int r8 = x / (D / 4), d = (x - r8 * (D / 4)) * 4, r = 8 * n + r8;
        if (r >= it.rows) continue;
        float mm = -CUDART_INF_F, ll = 0.0f, lw = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, red[w * R + r]);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float mw = red[w * R + r];
          if (mw == -CUDART_INF_F) continue;
          const float f = ex2(mw - mm);
          ll = fmaf(f, red[(WARPS + w) * R + r], ll);
          lw = fmaf(f, red[(2 * WARPS + w) * R + r], lw);
          const float4 v = *reinterpret_cast<const float4*>(join + (w * 8 + r8) * C::RED_LD + d);
          acc.x = fmaf(f, v.x, acc.x); acc.y = fmaf(f, v.y, acc.y);
          acc.z = fmaf(f, v.z, acc.z); acc.w = fmaf(f, v.w, acc.w);
        }
        acc.x += lw; acc.y += lw; acc.z += lw; acc.w += lw;
        if (it.whole) {
          const int rr = it.rt * R + r, i = rr / p.G, hq = it.h * p.G + rr - i * p.G;
          const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
          store_out(p, (it.sq.tok0 + i) * p.ldo + (long long)hq * D + d,
                    make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
          if (p.lse && d == 0)
            p.lse[(it.sq.tok0 + i) * p.Hq + hq] = ll == 0.0f ? -CUDART_INF_F : (mm + log2f(ll)) * 0.6931471805599453f;
        } else {
          *reinterpret_cast<float4*>(out + r * D + d) = acc;
          if (d == 0) {
            out[R * D + r] = mm;
            out[R * D + R + r] = ll;
          }
        }
      }
    }
    if (it.more) cut = make_int4(it.b, it.item, 1 + it.more, 0);
    have = more && !dead;
    it = nx;
    if (have) __syncthreads();                   // join and red are written again
  }
  if (tid == 0) p.cut[blockIdx.x] = cut;
  if (dead) {                                    // copies that may still be in flight (none otherwise)
    for (uint32_t u = use; u < use + NS; ++u) mbar_wait_bounded(&full[u % NS], u / NS & 1u, nullptr, 1000000ull);
  }
}

// Query rows of one head that a CTA takes at once: the eight columns of an n-tile times NT.
int row_tiles(int D, long long rows) { return rows <= 8 ? 1 : (rows <= 16 || D != 64 ? 2 : 4); }

template <typename F>
void with_shape(int D, int nt, F&& f) {
  auto go = [&](auto d) {
    constexpr int DD = decltype(d)::value;
    if (nt == 1) f(d, std::integral_constant<int, 1>{});
    else if (nt == 2 || DD != 64) f(d, std::integral_constant<int, 2>{});
    else if constexpr (DD == 64) f(d, std::integral_constant<int, 4>{});
  };
  if (D == 64) go(std::integral_constant<int, 64>{});
  else if (D == 128) go(std::integral_constant<int, 128>{});
  else go(std::integral_constant<int, 256>{});
}

}  // namespace kva

// Which kernel: many rows of a head at once are worth dequantizing a tile into shared memory for the
// large tensor-core tiles; this one streams the cache again for its most rows each. (Heads of 256
// do not fit the other's tensor memory with its two groups of rows.) Measured over 8 kv heads, in us, this one / the other: D = 128, 32
// sequences of 1024 tokens, 16 rows a head 25 / 57, 32 rows 57 / 57, 64 rows 129 / 59; 8 of 2048, 16 rows
// 23 / 37, 32 rows 47 / 37; one of 8192, 16 rows 23 / 31, 32 rows 45 / 31. D = 64, 32 of 1024: 32 rows 31 / 45, 48
// rows 70 / 45; one of 8192: 32 rows 30 / 27.
static bool many_rows(int D, long long rows) { return D != 256 && rows > (D == 64 ? 32 : 16); }
// fp16 outputs over few keys stay with this kernel for any number of rows. The other one rounds k, v and the
// probabilities to fp16, each as coarsely as the output itself is rounded, and over few keys nothing averages
// that. Error against 64 bits, in units of the output's rounding, this one / the other: up to 128 keys (whole
// caches or windows) 1.0 / 1.2 to 1.68, at 200 to 400 1.0 / 1.2 to 1.45, at 1000 1.0 / 1.1 to 1.27. In us, 4 sequences of 100 tokens, D = 128: 16 rows a
// token 23 / 23, 7 rows 30 / 25, 8 heads of 8 54 / 25; of 40 tokens 12 / 23, 13 / 25, 29 / 25. (bf16 rounds to 2^-8: 1.02 in either.)
constexpr int kFewKeys = 128;
static bool few_keys_f16(int dtype, long long keys, int causal, long long window) {
  return dtype == GPTQ_F16 && (keys <= kFewKeys || (causal && window > 0 && window <= kFewKeys));
}

size_t kv_attention_tc_workspace_bytes(int D);
gptq_status kv_attention_tc_launch(const kva::Params& p, int D, void* ws, cudaStream_t s);

// Workspace: per CTA the item it began and left, and two parts.
size_t kv_attention_workspace_bytes(long long total_q, int Hq, int H, int D, long long batch, long long max_q) {
  using namespace kva;
  (void)total_q;
  (void)batch;
  size_t bytes = 0;                              // of this kernel, and of the other where a call can take either
  with_shape(D, row_tiles(D, max_q * (Hq / H)), [&](auto d, auto n) {
    using C = Cfg<decltype(d)::value, decltype(n)::value>;
    const size_t ctas = (size_t)sm_count() * C::OCC;
    bytes = round256(16 * ctas) + ctas * 2 * C::PART * 4;
  });
  return many_rows(D, max_q * (Hq / H)) ? std::max(bytes, kv_attention_tc_workspace_bytes(D)) : bytes;
}

gptq_status kv_attention_launch(const void* Q, int dtype, long long total_q, int Hq, int H, int D, long long ldq,
                                const int* cu_q, const int* kv_lens, const int* table, long long ldt,
                                long long table_width, long long batch, long long max_q, const void* pool,
                                long long num_pages, int page, float sm_scale, int causal, long long window, void* O,
                                long long ldo, float* lse, void* ws, cudaStream_t s) {
  using namespace kva;
  Params p{};
  p.Q = Q; p.O = O; p.lse = lse; p.cu_q = cu_q; p.kv_lens = kv_lens; p.table = table;
  p.pool = reinterpret_cast<const uint8_t*>(pool);
  p.ldq = ldq; p.ldo = ldo; p.ldt = ldt; p.num_pages = num_pages;
  p.total_q = (int)total_q; p.max_q = (int)max_q; p.cap = (int)(table_width * page);
  p.Hq = Hq; p.H = H; p.G = Hq / H; p.batch = (int)batch; p.causal = causal; p.q_f16 = dtype == GPTQ_F16;
  set_pages(p, page);
  p.window = window > 0x7FFFFFFFLL ? 0 : window;         // every key is nearer than that; sums with it stay in range
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  if (many_rows(D, max_q * p.G) && !few_keys_f16(dtype, table_width * page, causal, window))
    return kv_attention_tc_launch(p, D, ws, s);
  gptq_status st = GPTQ_OK;
  with_shape(D, row_tiles(D, max_q * p.G), [&](auto d, auto n) {
    constexpr int DD = decltype(d)::value, NT = decltype(n)::value;
    using C = Cfg<DD, NT>;
    static PerDevice done[2];
    const auto kernel = p.q_f16 ? kv_split_kernel<DD, NT, true> : kv_split_kernel<DD, NT, false>;
    if ((st = allow_smem(done[p.q_f16], kernel, C::SMEM, "kv_split_kernel"))) return;
    const long long ctas = (long long)sm_count() * C::OCC;
    p.cut = reinterpret_cast<int4*>(ws);
    p.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + round256(16 * (size_t)ctas));
    kernel<<<(unsigned)ctas, THREADS, C::SMEM, s>>>(p, device_error_word());
    count_launch();
    if ((st = check_launch("kv_split_kernel"))) return;
    // nothing is cut when no item can be longer than kWholeTiles and every CTA gets at most one
    const long long row_items = (max_q * p.G + C::R - 1) / C::R;
    if (table_width * page <= kWholeTiles * TILE && batch * H * row_items <= ctas) return;
    launch_pdl(kv_join_kernel<DD, C::R>, dim3((unsigned)ctas, NT), dim3(JOIN_WARPS * 32), 0, s, p);
    count_launch();
    st = check_launch("kv_join_kernel");
  });
  return st;
}

}  // namespace gptq
