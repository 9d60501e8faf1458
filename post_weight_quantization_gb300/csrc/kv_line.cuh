// What the attention kernels over the 4-bit paged cache share: their parameters, the line of
// key tiles that is cut evenly over the CTAs, the copies of a tile, and the join of items that
// were cut. An item is one sequence's R query rows of one kv head; its tiles are 128 keys.
#pragma once

#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "elem.cuh"

namespace gptq {
namespace kva {

constexpr int TILE = 128;                       // keys of a tile
constexpr int kWholeTiles = 8;                  // items of up to so many tiles are not cut when every CTA has at most one
constexpr int SCAN = 128;                       // threads that sum the batch's units

struct Params {
  const void* Q;
  void* O;
  float* lse;
  const int* cu_q;
  const int* kv_lens;
  const int* table;
  const uint8_t* pool;
  long long ldq, ldo, ldt, num_pages;
  int total_q, max_q, cap;                      // query tokens, the most of a sequence; keys that a row of the table holds
  int Hq, H, G, page, batch, causal, q_f16;
  int pb, pb_log2;                              // keys of a block: the largest power of two up to TILE that divides page
  uint32_t page_mul;                            // ceil(2^32 / (page / pb)); 0 when page is pb
  long long window;
  float scale_log2;                             // sm_scale * log2(e)
  int4* cut;                                    // workspace, per CTA: {sequence, item, parts} of the item it begins and others end
  float* part;                                  // workspace: 2 x CTAs x (R x D values, R maxima, R sums)
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
// The power of two that brings a query row's largest value mx to [2^14, 2^15); 0 for a row of zeros and
// for one with an infinity, which stays one.
__device__ __forceinline__ int row_exponent(float mx) {
  const int e = 14 - ((int)(__float_as_uint(mx) >> 23) - 127);
  return mx == 0.0f || mx == CUDART_INF_F ? 0 : max(-126, min(126, e));
}
// One sequence of the batch, as the line of tiles sees it.
struct Seq {
  long long tok0;                // its first query token
  int nq, len;                   // query tokens, cached keys
  int t0, tiles, nrt;            // first tile, tiles of an item, row tiles of a head
  long long items;               // H * nrt
};

// Its tokens a ... z - 1 are in range (as unsigned numbers: negative ones are large).
__device__ __forceinline__ bool steps_ok(const Params& p, int a, int z) {
  return (unsigned)z <= (unsigned)p.total_q && (unsigned)a <= (unsigned)z;
}
// Steps out of range count as no tokens, more tokens than max_q, by which the host has chosen the
// launches, as max_q, and lengths are limited to theirs. find_start, which every CTA begins with, reports all three.
__device__ __forceinline__ Seq load_seq(const Params& p, int b, int R) {
  Seq s;
  const int a = p.cu_q[b], z = p.cu_q[b + 1], len = min(max(p.kv_lens[b], 0), p.cap);
  s.tok0 = a;
  s.nq = steps_ok(p, a, z) ? min(z - a, p.max_q) : 0;
  s.len = len;
  const long long lo = p.window > 0 ? (long long)len - s.nq - p.window + 1 : 0;
  s.t0 = lo > 0 ? (int)(lo / TILE) : 0;
  const int n = (s.len + TILE - 1) / TILE - s.t0;
  s.tiles = n > 0 ? n : 1;
  s.nrt = (int)(((long long)s.nq * p.G + R - 1) / R);
  s.items = (long long)p.H * s.nrt;
  return s;
}

__device__ __forceinline__ bool seq_ok(const Params& p, int b) {
  const int a = p.cu_q[b], z = p.cu_q[b + 1];
  return steps_ok(p, a, z) && z - a <= p.max_q && (unsigned)p.kv_lens[b] <= (unsigned)p.cap;
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

// Where the CTA starts on the line of items: sequence b, offset off in its units. Every CTA sums
// the batch's units itself (the lengths are on the device). An item is COST + tiles
// units; or one unit, and so never cut, when the items are short and every CTA gets at most
// one. Returns the units per CTA in `per`, all units in `total`.
template <int R, int COST>
__device__ __forceinline__ void find_start(const Params& p, long long* sh, long long& total, long long& per, int& b0,
                                           long long& off, bool& whole, int* err) {
  const int tid = threadIdx.x, nb = (p.batch + SCAN - 1) / SCAN;                 // the first SCAN threads scan
  long long units = 0, items = 0;
  int longest = 0;
  for (int k = 0; k < nb; ++k) {
    const int b = tid * nb + k;
    if (tid < SCAN && b < p.batch) {
      const Seq q = load_seq(p, b, R);
      if (!seq_ok(p, b)) report_device_error(err, DEVERR_INDEX);
      items += q.items;
      units += q.items * (q.tiles + COST);
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
  if ((tid & 31) == 31 && tid < SCAN) {
    sh[tid >> 5] = units;
    sh[4 + (tid >> 5)] = items;
    sh[8 + (tid >> 5)] = longest;
  }
  if (tid == 0) sh[12] = p.batch;                // no sequence unless one is found below
  __syncthreads();
  long long ub = 0, ib = 0, ut = 0, it = 0;
  for (int w = 0; w < SCAN / 32; ++w) {
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
  if (tid < SCAN && start >= at && start < at + mine) {              // exactly one thread when start < total
    for (int k = 0; k < nb; ++k) {
      const int b = tid * nb + k;
      const Seq q = load_seq(p, b, R);
      const long long u = whole ? q.items : q.items * (q.tiles + COST);
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

// A head's row tiles are taken from both ends in turn: under a causal mask the first rows see the fewest
// keys and the last the most, while the line counts every item's tiles alike. (A prompt of 4096 tokens, 64 + 8
// heads of 128: 543 us in order, 381 this way; 1024 tokens over 8187 keys 281, 268.)
__device__ __forceinline__ int row_tile(int k, int nrt) { return k & 1 ? nrt - 1 - (k >> 1) : k >> 1; }

// One item, or the part of it that a CTA takes.
struct Item {
  Seq sq;
  int b, item, h, rt, rows, i0, i1;
  int lo_all, hi_all;            // the keys that some row sees: lo_all ... hi_all - 1
  int tl, nt;                    // its tiles
  bool lead, whole;              // began in an earlier CTA; not cut at all
  int more;                      // CTAs after this one that hold parts of it
};

// The CTA's way along the line: next() gives its next item (false when there is none).
template <int R, int COST>
struct Line {
  long long left, off, per;      // units left, offset in sequence b's units, units of a CTA
  int b;
  bool one_each;                 // an item is one unit
  __device__ __forceinline__ void init(const Params& p, long long* sh, int* err) {
    long long total;
    find_start<R, COST>(p, sh, total, per, b, off, one_each, err);
    left = total - per * blockIdx.x;
    left = left < per ? left : per;
  }
  __device__ __forceinline__ bool next(const Params& p, Item& it) {
    while (left > 0 && b < p.batch) {
      it.sq = load_seq(p, b, R);
      const int cost = one_each ? 1 : it.sq.tiles + COST;
      if (off >= it.sq.items * cost) {
        ++b;
        off = 0;
        continue;
      }
      const long long item = off / cost;
      const int x = (int)(off - item * cost), y = (int)(left < cost - x ? x + left : cost);
      off += y - x;
      left -= y - x;
      const int ta = one_each ? 0 : max(0, x - COST), tb = one_each ? it.sq.tiles : max(0, y - COST);
      if (tb <= ta) continue;                    // only the item's beginning: its first tile is the next CTA's
      const Seq& q = it.sq;
      it.b = b;
      it.item = (int)item;
      it.h = it.item / q.nrt;
      it.rt = row_tile(it.item - it.h * q.nrt, q.nrt);
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
  }
};

// The copies of a tile: TILE / pb blocks of pb keys, each inside one page; a block is one copy
// where it is the whole page, else its K codes, V codes and numbers are one copy each. Lanes
// issue them, each its own: a copy costs its warp about 70 cycles.
struct Copies {
  int ncp, piece, part, tile_blocks, ppb;       // copies of a block; this lane's block and part; blocks of a tile, of a page
  __device__ __forceinline__ void init(const Params& p, int lane) {
    ppb = p.page >> p.pb_log2;
    ncp = ppb == 1 ? 1 : 3;
    piece = ncp == 1 ? lane : lane / 3;
    part = ncp == 1 ? 3 : lane - 3 * piece;
    tile_blocks = TILE >> p.pb_log2;
  }
  // where this lane's copy of the item's tile i starts (-1: no keys there)
  __device__ __forceinline__ long long source(const Params& p, const Item& it, int i, int D, int* err) const {
    const int jb = (it.tl + i) * tile_blocks + piece;
    if (piece >= tile_blocks || i >= it.nt || (jb << p.pb_log2) >= it.hi_all) return -1;
    const int idx = ppb == 1 ? jb : (int)__umulhi((uint32_t)jb, p.page_mul);
    int pg = p.table[it.b * p.ldt + idx];
    if (pg < 0 || pg >= p.num_pages) {
      report_device_error(err, DEVERR_INDEX);
      pg = 0;
    }
    const int at = (jb - idx * ppb) << p.pb_log2;                    // first token of the block in its page
    const long long block = (long long)p.page * (D + 8);
    return ((long long)pg * p.H + it.h) * block + (part == 3 ? 0LL : part == 2 ? (long long)p.page * D + at * 8
                                                                               : (long long)(part * p.page + at) * (D / 2));
  }
  // all of the tile's copies into `dst`, completing on `full` (whole warp)
  __device__ __forceinline__ void issue(const Params& p, uint32_t dst, uint64_t* full, long long src, int D, int lane) const {
    const unsigned copies = __popc(__ballot_sync(0xffffffffu, src >= 0));
    if (lane == 0) mbar_arrive_expect_tx(full, (ncp == 1 ? copies : copies / 3) * p.pb * (D + 8));
    __syncwarp();
    if (src >= 0) {
      dst += piece * p.pb * (D + 8);
      if (part == 3) bulk_load(dst, p.pool + src, p.pb * (D + 8), full);
      else if (part == 2) bulk_load(dst + p.pb * D, p.pool + src, p.pb * 8, full);
      else bulk_load(dst + part * p.pb * (D / 2), p.pool + src, p.pb * (D / 2), full);
    }
  }
};

// Joins the parts of the items that were cut. CTA (c, y) takes the item that CTA c of the other
// kernel began and others ended; its parts lie in c's second place and the following CTAs' first.
// A warp takes a row, all its parts in flight together; where there are many parts, two to eight
// warps share a row.
constexpr int JOIN_WARPS = 16;
template <int D, int R>
__global__ void __launch_bounds__(JOIN_WARPS * 32) kv_join_kernel(Params p) {
  constexpr int VPL = D / 32, PART = R * D + 2 * R;
  using V = typename std::conditional<VPL == 2, float2, float4>::type;       // a lane's values, NV vectors of VW
  constexpr int NV = VPL == 2 ? 1 : VPL / 4, VW = VPL / NV;
  __shared__ float sl[JOIN_WARPS], so[JOIN_WARPS][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  const int c = blockIdx.x;
  const int4 cut = p.cut[c];
  if (cut.z == 0) return;
  const Seq sq = load_seq(p, cut.x, R);
  const int h = cut.y / sq.nrt, rt = row_tile(cut.y - h * sq.nrt, sq.nrt), np = cut.z;
  const long long all_rows = (long long)sq.nq * p.G;
  auto part_of = [&](int k) { return p.part + (2LL * (c + k) + (k == 0 ? 1 : 0)) * PART; };
  float mm, ll, acc[VPL];
  auto largest = [&](int r) {
    mm = -CUDART_INF_F;
    for (int k = lane; k < np; k += 32) mm = fmaxf(mm, part_of(k)[R * D + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    ll = 0.0f;
#pragma unroll
    for (int k = 0; k < VPL; ++k) acc[k] = 0.0f;
  };
  auto add = [&](int k, int r) {
    const float* pt = part_of(k);
    const float mk = pt[R * D + r], f = mk == -CUDART_INF_F ? 0.0f : ex2(mk - mm);
    ll = fmaf(f, pt[R * D + R + r], ll);
#pragma unroll
    for (int x = 0; x < NV; ++x) {               // lane's values: VW at (32 x + lane) VW
      const V v = *reinterpret_cast<const V*>(pt + r * D + (32 * x + lane) * VW);
      const float* vf = reinterpret_cast<const float*>(&v);
#pragma unroll
      for (int y = 0; y < VW; ++y) acc[x * VW + y] = fmaf(f, vf[y], acc[x * VW + y]);
    }
  };
  auto write = [&](int rr) {
    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
    const int i = rr / p.G, hq = h * p.G + rr - i * p.G;
    const long long at = (sq.tok0 + i) * p.ldo + (long long)hq * D;
#pragma unroll
    for (int x = 0; x < VPL; ++x) {
      float v = acc[x] * inv;
      const long long d = at + (32 * (x / VW) + lane) * VW + x % VW;
      if (p.q_f16) {
        v = v == v ? fminf(fmaxf(v, -65504.0f), 65504.0f) : v;
        reinterpret_cast<__half*>(p.O)[d] = __float2half_rn(v);
      } else {
        reinterpret_cast<__nv_bfloat16*>(p.O)[d] = __float2bfloat16_rn(v);
      }
    }
    if (p.lse && lane == 0)
      p.lse[(sq.tok0 + i) * p.Hq + hq] = ll == 0.0f ? -CUDART_INF_F : (mm + log2f(ll)) * 0.6931471805599453f;
  };
  if (np <= 4) {
    for (int r = JOIN_WARPS * blockIdx.y + warp; r < R && (long long)rt * R + r < all_rows; r += JOIN_WARPS * gridDim.y) {
      float mk[4], lk[4];
      V vk[4][NV];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        mk[k] = -CUDART_INF_F;
        if (k < np) {
          const float* pt = part_of(k);
          mk[k] = pt[R * D + r];
          lk[k] = pt[R * D + R + r];
#pragma unroll
          for (int x = 0; x < NV; ++x) vk[k][x] = *reinterpret_cast<const V*>(pt + r * D + (32 * x + lane) * VW);
        }
      }
      mm = fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3]));
      ll = 0.0f;
#pragma unroll
      for (int k = 0; k < VPL; ++k) acc[k] = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (mk[k] == -CUDART_INF_F) continue;
        const float f = ex2(mk[k] - mm);
        ll = fmaf(f, lk[k], ll);
#pragma unroll
        for (int x = 0; x < VPL; ++x) acc[x] = fmaf(f, reinterpret_cast<const float*>(vk[k])[x], acc[x]);
      }
      write(rt * R + r);
    }
    return;
  }
  const long long rows = all_rows - (long long)rt * R;
  const int rp = rows <= 2 ? 2 : rows <= 4 ? 4 : 8, share = JOIN_WARPS / rp, slot = warp & (rp - 1), s0 = warp / rp;
  for (int r0 = rp * blockIdx.y; r0 < R && r0 < rows; r0 += rp * gridDim.y) {
    const int r = r0 + slot;
    const bool live = r < rows;
    if (live) {
      largest(r);
#pragma unroll 8
      for (int k = s0; k < np; k += share) add(k, r);
    }
    if (s0 && live) {
      if (lane == 0) sl[warp] = ll;
#pragma unroll
      for (int x = 0; x < VPL; ++x) so[warp][(32 * (x / VW) + lane) * VW + x % VW] = acc[x];
    }
    __syncthreads();
    if (!s0 && live) {
      for (int w = slot + rp; w < JOIN_WARPS; w += rp) {
        ll += sl[w];
#pragma unroll
        for (int x = 0; x < VPL; ++x) acc[x] += so[w][(32 * (x / VW) + lane) * VW + x % VW];
      }
      write(rt * R + r);
    }
    __syncthreads();
  }
}

// The page geometry of a call (host).
inline void set_pages(Params& p, int page) {
  p.page = page;
  p.pb_log2 = 4;
  while (p.pb_log2 < 7 && page % (2 << p.pb_log2) == 0) ++p.pb_log2;
  p.pb = 1 << p.pb_log2;
  const unsigned ppb = (unsigned)(page >> p.pb_log2);
  p.page_mul = ppb == 1 ? 0u : (uint32_t)((0x100000000ULL + ppb - 1) / ppb);
}

inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace kva
}  // namespace gptq
