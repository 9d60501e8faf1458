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
//     2^-11 of each, random in sign, against the output's own 2^-8 or 2^-11. They are
//     brought to the top of fp16's range by a power of two that follows the largest V scale
//     seen, so small probabilities keep their bits down to 2^-24 of the largest.
//   Why mma.sync and not tcgen05: the product is bound by HBM bandwidth (one pass over the
//   cache for at most 32 rows), and tcgen05 would need the codes unpacked to 16 bits in
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
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "elem.cuh"

namespace gptq {
namespace kva {

constexpr int WARPS = 4, THREADS = WARPS * 32;
constexpr int KC = 32;                          // keys of a warp's chunk
constexpr int TILE = WARPS * KC;                // keys of a tile
constexpr int kItemCost = 2;                    // what beginning an item costs, in tiles
constexpr int kWholeTiles = 8;                  // items of up to so many tiles are not cut when every CTA has at most one
constexpr float kSlack = 6.0f;                  // a row's maximum may lag by 2^6 before it is moved
constexpr int kVExp = 8;                        // V scales are brought below 2^(kVExp + 1)

struct Params {
  const void* Q;
  void* O;
  float* lse;
  const int* cu_q;
  const int* kv_lens;
  const int* table;
  const uint8_t* pool;
  long long ldq, ldo, ldt, total_q, table_width, num_pages;
  int Hq, H, G, page, batch, causal, q_f16;
  int pb, pb_log2;                              // keys of a block: the largest power of two up to TILE that divides page
  uint32_t page_mul;                            // ceil(2^32 / (page / pb)); 0 when page is pb
  long long window;
  float scale_log2;                             // sm_scale * log2(e)
  int4* cut;                                    // workspace, per CTA: {sequence, item, parts} of the item it begins and others end
  float* part;                                  // workspace: 2 x CTAs x (R x D values, R maxima, R sums)
};

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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
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
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126 ... 127
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

// One sequence of the batch, as the line of tiles sees it.
struct Seq {
  long long tok0;                // its first query token
  int nq, len;                   // query tokens, cached keys
  int t0, tiles, nrt;            // first tile, tiles of an item, row tiles of a head
  long long items;               // H * nrt
};

__device__ __forceinline__ Seq load_seq(const Params& p, int b, int R, int* err) {
  Seq s;
  long long a = p.cu_q[b], z = p.cu_q[b + 1], len = p.kv_lens[b];
  const long long cap = p.table_width * p.page;
  if (a < 0 || z > p.total_q || len < 0 || len > cap) {
    report_device_error(err, DEVERR_INDEX);
    a = a < 0 ? 0 : a;
    z = z > p.total_q ? p.total_q : z;
    len = len < 0 ? 0 : (len > cap ? cap : len);
  }
  s.tok0 = a;
  s.nq = z > a ? (int)(z - a) : 0;
  s.len = (int)len;
  const long long lo = p.window > 0 ? len - s.nq - p.window + 1 : 0;
  s.t0 = lo > 0 ? (int)(lo / TILE) : 0;
  const int n = (s.len + TILE - 1) / TILE - s.t0;
  s.tiles = n > 0 ? n : 1;
  s.nrt = (int)(((long long)s.nq * p.G + R - 1) / R);
  s.items = (long long)p.H * s.nrt;
  return s;
}

__device__ __forceinline__ void store_out(const Params& p, long long at, float4 v) {
  if (p.q_f16) {
    const float lim = 65504.0f;
    v.x = v.x == v.x ? fminf(fmaxf(v.x, -lim), lim) : v.x;
    v.y = v.y == v.y ? fminf(fmaxf(v.y, -lim), lim) : v.y;
    v.z = v.z == v.z ? fminf(fmaxf(v.z, -lim), lim) : v.z;
    v.w = v.w == v.w ? fminf(fmaxf(v.w, -lim), lim) : v.w;
    *reinterpret_cast<uint2*>(reinterpret_cast<__half*>(p.O) + at) = make_uint2(pack_half2(v.x, v.y), pack_half2(v.z, v.w));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.O) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
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

template <int D, int NT, bool MASK>
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
    uint32_t b[NT][2];
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
        b[n][e] = movmatrix(pack_half2(pc[0], pc[1]));
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
        for (int n = 0; n < NT; ++n)
          mma_f16(st.o[4 * w + by][n], l2 & 0x000F000Fu, l2 & 0x00F000F0u, h2 & 0x000F000Fu, h2 & 0x00F000F0u, b[n][0],
                  b[n][1]);
      }
  }
}



// Where the CTA starts on the line of items: sequence b, offset off in its units. Every CTA sums
// the batch's units itself (the lengths are on the device). An item is kItemCost + tiles
// units; or one unit, and so never cut, when the items are short and every CTA gets at most
// one. Returns the units per CTA in `per`, all units in `total`.
template <int R>
__device__ __forceinline__ void find_start(const Params& p, long long* sh, long long& total, long long& per, int& b0,
                                           long long& off, bool& whole, int* err) {
  const int tid = threadIdx.x, nb = (p.batch + THREADS - 1) / THREADS;
  long long units = 0, items = 0;
  int longest = 0;
  for (int k = 0; k < nb; ++k) {
    const int b = tid * nb + k;
    if (b < p.batch) {
      const Seq q = load_seq(p, b, R, err);
      items += q.items;
      units += q.items * (q.tiles + kItemCost);
      if (q.items) longest = max(longest, q.tiles);
    }
  }
  const long long my_units = units, my_items = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, units, o), i = __shfl_up_sync(0xffffffffu, items, o);
    if ((tid & 31) >= o) { units += u; items += i; }
    longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  }
  if ((tid & 31) == 31) {
    sh[tid >> 5] = units;
    sh[4 + (tid >> 5)] = items;
    sh[8 + (tid >> 5)] = longest;
  }
  if (tid == 0) sh[12] = p.batch;                // no sequence unless one is found below
  __syncthreads();
  long long ub = 0, ib = 0, ut = 0, it = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w < (tid >> 5)) { ub += sh[w]; ib += sh[4 + w]; }
    ut += sh[w];
    it += sh[4 + w];
    longest = max(longest, (int)sh[8 + w]);
  }
  whole = longest <= kWholeTiles && it <= gridDim.x;
  total = whole ? it : ut;
  per = whole ? 1 : (ut + gridDim.x - 1) / gridDim.x;
  const long long mine = whole ? my_items : my_units, start = per * blockIdx.x;
  long long at = whole ? ib + items - my_items : ub + units - my_units;   // units before this thread's sequences
  if (start >= at && start < at + mine) {        // exactly one thread when start < total
    for (int k = 0; k < nb; ++k) {
      const int b = tid * nb + k;
      const Seq q = load_seq(p, b, R, err);
      const long long u = whole ? q.items : q.items * (q.tiles + kItemCost);
      if (start < at + u) {
        sh[12] = b;
        sh[13] = start - at;
        break;
      }
      at += u;
    }
  }
  __syncthreads();
  b0 = (int)sh[12];
  off = sh[13];
}

// One item, or the part of it that a CTA takes.
struct Item {
  Seq sq;
  int b, item, h, rt, rows, i0, i1;
  int lo_all, hi_all;            // the keys that some row sees: lo_all ... hi_all - 1
  int tl, nt;                    // its tiles
  bool lead, whole;              // began in an earlier CTA; not cut at all
  int more;                      // CTAs after this one that hold parts of it
};

template <int D, int NT>
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
  long long total, per, off;
  int b;
  bool one_each;
  find_start<R>(p, sh, total, per, b, off, one_each, err);
  grid_dep_launch();
  long long left = total - per * blockIdx.x;
  left = left < per ? left : per;
  const long long block = (long long)p.page * (D + 8), page_step = (long long)p.H * block;
  const int ppb = p.page >> p.pb_log2;           // blocks of a page
  // where this warp's two 16-key tiles lie in a stage: codes and numbers
  uint32_t koff[2], noff[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int k = warp * KC + 16 * m, blk = k >> p.pb_log2, at = k & (p.pb - 1);
    koff[m] = blk * p.pb * (D + 8) + at * (D / 2);
    noff[m] = blk * p.pb * (D + 8) + p.pb * D + at * 8;
  }

  // The next item of this CTA (false when there is none): takes its units off the line.
  auto next_item = [&](Item& it) -> bool {
    while (left > 0 && b < p.batch) {
      it.sq = load_seq(p, b, R, err);
      const int cost = one_each ? 1 : it.sq.tiles + kItemCost;
      if (off >= it.sq.items * cost) {
        ++b;
        off = 0;
        continue;
      }
      const long long item = off / cost;
      const int x = (int)(off - item * cost), y = (int)(left < cost - x ? x + left : cost);
      off += y - x;
      left -= y - x;
      const int ta = one_each ? 0 : max(0, x - kItemCost), tb = one_each ? it.sq.tiles : max(0, y - kItemCost);
      if (tb <= ta) continue;                    // only the item's beginning: its first tile is the next CTA's
      const Seq& q = it.sq;
      it.b = b;
      it.item = (int)item;
      it.h = it.item / q.nrt;
      it.rt = it.item - it.h * q.nrt;
      const long long rest = (long long)q.nq * p.G - (long long)it.rt * R;
      it.rows = (int)(rest < R ? rest : R);
      it.i0 = it.rt * R / p.G;
      it.i1 = (it.rt * R + it.rows - 1) / p.G;
      it.lead = ta > 0;
      it.whole = ta == 0 && tb == q.tiles;
      it.more = it.whole || it.lead ? 0 : (int)((cost - y + per - 1) / per);
      const int pos0 = q.len - q.nq;             // position of the sequence's first query token
      const long long klo = p.window > 0 ? (long long)pos0 + it.i0 - p.window + 1 : 0;
      it.lo_all = klo > 0 ? (int)klo : 0;
      it.hi_all = p.causal ? min(q.len, max(0, pos0 + it.i1 + 1)) : q.len;
      it.tl = max(q.t0 + ta, it.lo_all / TILE);
      it.nt = max(0, min(q.t0 + tb, (it.hi_all + TILE - 1) / TILE) - it.tl);
      return true;
    }
    return false;
  };

  // A tile is TILE / pb blocks of pb keys, each inside one page; a block is one copy where it
  // is the whole page, else its K codes, V codes and numbers are one copy each. Lanes issue
  // them, each its own, in the warp whose turn it is (tile i of the item is warp i % WARPS's):
  // a copy costs its warp about 70 cycles.
  const int ncp = ppb == 1 ? 1 : 3, piece = ncp == 1 ? lane : lane / 3, cpart = ncp == 1 ? 3 : lane - 3 * piece;
  const int tile_blocks = TILE >> p.pb_log2;
  bool dead = false;
  // where this lane's copy of tile i starts (-1: no keys there)
  auto source = [&](const Item& it, int i) -> long long {
    const int jb = (it.tl + i) * tile_blocks + piece;
    if (piece >= tile_blocks || i >= it.nt || (jb << p.pb_log2) >= it.hi_all) return -1;
    const int idx = ppb == 1 ? jb : (int)__umulhi((uint32_t)jb, p.page_mul);
    int pg = p.table[it.b * p.ldt + idx];
    if (pg < 0 || pg >= p.num_pages) {
      report_device_error(err, DEVERR_INDEX);
      pg = 0;
    }
    const int at = (jb - idx * ppb) << p.pb_log2;                    // first token of the block in its page
    return pg * page_step + it.h * block + (cpart == 3 ? 0LL : cpart == 2 ? (long long)p.page * D + at * 8
                                                                         : (long long)(cpart * p.page + at) * (D / 2));
  };
  auto issue = [&](uint32_t u, long long src) {
    const uint32_t st = u % NS;
    if (!mbar_wait_poll(&empty[st], (u / NS & 1u) ^ 1u, nullptr)) {
      if (lane == 0) report_device_error(err, DEVERR_TIMEOUT);
      dead = true;
      return;
    }
    const unsigned copies = __popc(__ballot_sync(0xffffffffu, src >= 0));
    if (lane == 0) mbar_arrive_expect_tx(&full[st], (ncp == 1 ? copies : copies / 3) * p.pb * (D + 8));
    __syncwarp();
    if (src >= 0) {
      const uint32_t dst = ring + st * C::STAGE + piece * p.pb * (D + 8);
      if (cpart == 3) bulk_load(dst, p.pool + src, p.pb * (D + 8), &full[st]);
      else if (cpart == 2) bulk_load(dst + p.pb * D, p.pool + src, p.pb * 8, &full[st]);
      else bulk_load(dst + cpart * p.pb * (D / 2), p.pool + src, p.pb * (D / 2), &full[st]);
    }
  };

  uint32_t slot = 0, phase = 0;                  // the ring's next tile
  uint32_t use = 0;                              // tiles taken from the ring so far, through all items
  Item it;
  bool have = next_item(it);
  int4 cut = make_int4(0, 0, 0, 0);
  if (have && warp < NS - 1 && warp < it.nt) issue(use + warp, source(it, warp));

  while (have) {
    // this warp's next tile to issue, NS - 1 tiles before it is taken
    int ni = warp < NS - 1 ? warp + WARPS : warp;
    long long nsrc = source(it, ni);
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
          sum += v[k];
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      int e = 14 - ((int)(__float_as_uint(mx) >> 23) - 127);
      e = mx == 0.0f || mx > 3.0e38f ? 0 : max(-126, min(126, e));
      const float f = pow2(e);
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        float v[8];
        if (p.q_f16) unpack8<F16>(&raw[w], v); else unpack8<BF16>(&raw[w], v);
        st.q[n][4 * w] = pack_half2(v[0] * f, v[4] * f);
        st.q[n][4 * w + 1] = pack_half2(v[1] * f * 0.0625f, v[5] * f * 0.0625f);
        st.q[n][4 * w + 2] = pack_half2(v[2] * f, v[6] * f);
        st.q[n][4 * w + 3] = pack_half2(v[3] * f * 0.0625f, v[7] * f * 0.0625f);
      }
      const float rs = sum * f, rc = p.scale_log2 * pow2(-e);
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
        nsrc = source(it, ni);
      }
      if (!mbar_wait_bounded(&full[slot], phase, nullptr)) {
        if (lane == 0) report_device_error(err, DEVERR_TIMEOUT);
        dead = true;
      }
      const uint32_t base = ring + slot * C::STAGE;
      const int key0 = (it.tl + i) * TILE + warp * KC;
      if (i >= plain_lo && i <= plain_hi)
        chunk<D, NT, false>(st, base + koff[0], base + koff[1], base + noff[0], base + noff[1], p.pb, key0, g, t);
      else if (key0 < it.hi_all && key0 + KC > it.lo_all)
        chunk<D, NT, true>(st, base + koff[0], base + koff[1], base + noff[0], base + noff[1], p.pb, key0, g, t);
      __syncwarp();                              // every lane has read its part of the stage
      if (lane == 0) mbar_arrive(&empty[slot]);
      ++use;
      if (++slot == NS) {
        slot = 0;
        phase ^= 1u;
      }
    }

    // ---- the next item's first tiles are on their way while the warps meet over this one
    Item nx;
    const bool more = next_item(nx);
    if (more && !dead && warp < NS - 1 && warp < nx.nt) issue(use + warp, source(nx, warp));

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

// Joins the parts of the items that were cut: a CTA per (CTA c of the other kernel, n-tile)
// takes the item that c began and others ended, two warps per query row. The parts lie in
// c's second place and the following CTAs' first.
constexpr int JOIN_WARPS = 16;
template <int D, int NT>
__global__ void __launch_bounds__(JOIN_WARPS * 32) kv_join_kernel(Params p, int* __restrict__ err) {
  using C = Cfg<D, NT>;
  constexpr int R = C::R, VPL = D / 32;
  __shared__ float sl[JOIN_WARPS], so[JOIN_WARPS / 2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = warp >> 3;
  grid_dep_wait();
  const int c = blockIdx.x;
  const int4 cut = p.cut[c];
  if (cut.z == 0) return;
  const Seq sq = load_seq(p, cut.x, R, err);
  const int h = cut.y / sq.nrt, rt = cut.y - h * sq.nrt, r = 8 * blockIdx.y + (warp & 7), rr = rt * R + r;
  const bool live = rr < (long long)sq.nq * p.G;
  const int np = cut.z;
  auto part_of = [&](int k) { return p.part + (2LL * (c + k) + (k == 0 ? 1 : 0)) * C::PART; };
  float mm = -CUDART_INF_F, ll = 0.0f, acc[VPL];
#pragma unroll
  for (int k = 0; k < VPL; ++k) acc[k] = 0.0f;
  if (live) {
    for (int k = lane; k < np; k += 32) mm = fmaxf(mm, part_of(k)[R * D + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
#pragma unroll 8
    for (int k = half; k < np; k += 2) {
      const float* pt = part_of(k);
      const float mk = pt[R * D + r], f = mk == -CUDART_INF_F ? 0.0f : ex2(mk - mm);
      ll = fmaf(f, pt[R * D + R + r], ll);
#pragma unroll
      for (int x = 0; x < VPL; ++x) acc[x] = fmaf(f, pt[r * D + lane * VPL + x], acc[x]);
    }
  }
  if (half) {
    if (lane == 0) sl[warp & 7] = ll;
#pragma unroll
    for (int x = 0; x < VPL; ++x) so[warp & 7][lane * VPL + x] = acc[x];
  }
  __syncthreads();
  if (half || !live) return;
  ll += sl[warp];
  const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
  const int i = rr / p.G, hq = h * p.G + rr - i * p.G;
#pragma unroll
  for (int x = 0; x < VPL; ++x) {
    float v = (acc[x] + so[warp][lane * VPL + x]) * inv;
    const long long at = (sq.tok0 + i) * p.ldo + (long long)hq * D + lane * VPL + x;
    if (p.q_f16) {
      v = v == v ? fminf(fmaxf(v, -65504.0f), 65504.0f) : v;
      reinterpret_cast<__half*>(p.O)[at] = __float2half_rn(v);
    } else {
      reinterpret_cast<__nv_bfloat16*>(p.O)[at] = __float2bfloat16_rn(v);
    }
  }
  if (p.lse && lane == 0)
    p.lse[(sq.tok0 + i) * p.Hq + hq] = ll == 0.0f ? -CUDART_INF_F : (mm + log2f(ll)) * 0.6931471805599453f;
}

// Query rows of one head that a CTA takes at once: the eight columns of an n-tile times NT.
int row_tiles(int D, long long rows) { return rows <= 8 ? 1 : (rows <= 16 || D == 256 ? 2 : 4); }

template <typename F>
void with_shape(int D, int nt, F&& f) {
  auto go = [&](auto d) {
    constexpr int DD = decltype(d)::value;
    if (nt == 1) f(d, std::integral_constant<int, 1>{});
    else if (nt == 2 || DD == 256) f(d, std::integral_constant<int, 2>{});
    else if constexpr (DD != 256) f(d, std::integral_constant<int, 4>{});
  };
  if (D == 64) go(std::integral_constant<int, 64>{});
  else if (D == 128) go(std::integral_constant<int, 128>{});
  else go(std::integral_constant<int, 256>{});
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace kva

// Workspace: per CTA the item it began and left, and two parts.
size_t kv_attention_workspace_bytes(long long total_q, int Hq, int H, int D, long long batch, long long max_q) {
  using namespace kva;
  (void)total_q;
  (void)batch;
  size_t bytes = 0;
  with_shape(D, row_tiles(D, max_q * (Hq / H)), [&](auto d, auto n) {
    using C = Cfg<decltype(d)::value, decltype(n)::value>;
    const size_t ctas = (size_t)sm_count() * C::OCC;
    bytes = round256(16 * ctas) + ctas * 2 * C::PART * 4;
  });
  return bytes;
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
  p.ldq = ldq; p.ldo = ldo; p.ldt = ldt; p.total_q = total_q; p.table_width = table_width; p.num_pages = num_pages;
  p.Hq = Hq; p.H = H; p.G = Hq / H; p.page = page; p.batch = (int)batch; p.causal = causal; p.q_f16 = dtype == GPTQ_F16;
  p.pb_log2 = 4;
  while (p.pb_log2 < 7 && page % (2 << p.pb_log2) == 0) ++p.pb_log2;
  p.pb = 1 << p.pb_log2;
  const unsigned ppb = (unsigned)(page >> p.pb_log2);
  p.page_mul = ppb == 1 ? 0u : (uint32_t)((0x100000000ULL + ppb - 1) / ppb);
  p.window = window;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  gptq_status st = GPTQ_OK;
  with_shape(D, row_tiles(D, max_q * p.G), [&](auto d, auto n) {
    constexpr int DD = decltype(d)::value, NT = decltype(n)::value;
    using C = Cfg<DD, NT>;
    static bool attr_done = false;
    if (!attr_done) {
      if (cudaFuncSetAttribute(kv_split_kernel<DD, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) {
        st = set_error(GPTQ_ERR_CUDA, "cudaFuncSetAttribute(kv_split_kernel) failed");
        return;
      }
      attr_done = true;
    }
    const long long ctas = (long long)sm_count() * C::OCC;
    p.cut = reinterpret_cast<int4*>(ws);
    p.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + round256(16 * (size_t)ctas));
    kv_split_kernel<DD, NT><<<(unsigned)ctas, THREADS, C::SMEM, s>>>(p, device_error_word());
    count_launch();
    if ((st = check_launch("kv_split_kernel"))) return;
    // nothing is cut when no item can be longer than kWholeTiles and every CTA gets at most one
    const long long row_items = (max_q * p.G + C::R - 1) / C::R;
    if (table_width * page <= kWholeTiles * TILE && batch * H * row_items <= ctas) return;
    launch_pdl(kv_join_kernel<DD, NT>, dim3((unsigned)ctas, NT), dim3(JOIN_WARPS * 32), 0, s, p, device_error_word());
    count_launch();
    st = check_launch("kv_join_kernel");
  });
  return st;
}

}  // namespace gptq
