// Attention of many query rows per sequence and kv head over the 4-bit paged cache (a prompt's
// piece, wide head groups), on the 5th-generation tensor cores.
//
//   o_i = sum_j p_ij v_j,   p_i = softmax over the seen j of sm_scale * q_i . k_j
//
// An item is 256 query rows of one kv head as two groups of 128; keys and values of a tile of 128
// are dequantized once for both. Per tile and group two products of 128 x 128 x D:
//   S = Q K^T    Q and K in shared memory (fp16, K-major), S in tensor memory
//   O += P V     P from tensor memory (fp16, over S's own columns), V in shared memory as it was
//                dequantized (keys as rows: the MN-major B operand), O in tensor memory
// Roundings to fp16 (11 bits): k and v as code * scale + low, once (half of 2^-11, random, where the
// output type itself rounds to 2^-8 or 2^-11; measured in units of that rounding, the error against 64 bits is
// at most 1.04 for bf16 outputs; for fp16 ones 1.1 to 1.45 over values with a mean, which errors average
// out against, and 2.0 to 2.4 over values without one; up to 128 keys the other kernel takes those, with 1.0); the probabilities, 2^8 times too large, so that
// those down to 2^-22 of a row's largest keep all bits (a maximum that lags leaves them more). Queries are scaled by a power of two per
// row as in the other kernel, so bf16 ones are exact. Scores, maxima and sums are fp32.
// Keys past the end are zero, keys with a NaN among their numbers get a NaN k and a zero v, so a
// row sees the NaN in its score exactly when it sees the key.
//
//   warp 0        copies of the packed tiles (bulk copies into a ring of two)
//   warp 1        MMA issuer: the first tile's S; then per half tile and group P V, S of the next but one
//   warps 4-11    dequantize: half a key per thread, K then V, into a ring of three 128 x D buffers
//   warps 12-19   softmax: a query row per thread (four warps per group); at the item's end O
// Scores come by half tiles of 64 keys into the two halves of a group's columns: while the softmax
// works on one half, the MMAs bring the other (whole tiles, whose P lies over all of S, made the two
// take turns: 288 instead of 269 us). One pass over the scores: they are read from tensor memory 32 at
// a time and leave as probabilities from the maximum so far. (Two threads per row, which tell each
// other their maxima, took 341 us with half tiles: what is done per half tile then counts twice.)
// Bound: the tensor cores' 4 rows keys D operations; measured, 1024 tokens over 8187 keys, 64 + 8 heads of
// 128: 257 us, the call with the join 267 us, 49 % of the measured bf16 rate (with row tiles in order: 269
// and 279). Per 256 rows and 128 keys it takes 3700 cycles, of which 2048 are MMAs; the softmax warps' own
// latency is the rest.
// The tiles of all items form a line that is cut evenly over one CTA per SM, as in the other
// kernel, and cut items are joined afterwards.
#include "kv_line.cuh"

namespace gptq {
namespace kva {
namespace tc {

constexpr int R = 256, DEQ0 = 4, NDEQ = 8, SOFT0 = DEQ0 + NDEQ, THREADS = (SOFT0 + 8) * 32;
constexpr int kItemCost = 1;
constexpr int CH = 32;                          // scores a thread takes from tensor memory at once
constexpr float kSlack = 7.0f;                  // a row's maximum may lag by 2^7 before it is moved: probabilities stay below 2^15
constexpr float kShift = 8.0f;                  // probabilities are kept 2^kShift times too large
constexpr int REG_ISSUE = 72, REG_DEQ = 64, REG_SOFT = 136;       // 128 x 72 + 256 x 64 + 256 x 136, below 640 x 96

template <int D>
struct Cfg {
  static constexpr int BOXES = D / 64;          // 64-value columns of a row (128 bytes, one swizzle row)
  static constexpr int BOX = 128 * 128;         // bytes of a box of 128 rows
  static constexpr int MAT = BOXES * BOX;       // a 128 x D fp16 matrix
  static constexpr int STAGE = TILE * (D + 8);
  static constexpr int NC = 2, NM = 3;          // ring of packed tiles, ring of dequantized matrices
  static constexpr int CODES = 2 * MAT, MATS = CODES + (NC * STAGE + 1023) / 1024 * 1024, BARS = MATS + NM * MAT;
  static constexpr int SMEM = BARS + 512 + 1024;
  static constexpr int PART = R * D + 2 * R;
};

__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit_by(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t l;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(l));
  return l;
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Eight codes of a word as four fp16 pairs code * scale + low, one rounding each. 0x6400 | c is
// 1024 + c, less 1024 exactly c; codes in bits 4 to 7 come as 16 c. Pair i holds codes i and i + 4:
// queries are laid out alike, and the output's columns are put back at its end.
__device__ __forceinline__ uint4 dequant8(uint32_t w, __half2 scale, __half2 low) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = ((i < 2 ? w : w >> 8) & (i & 1 ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
    const __half2 a = *reinterpret_cast<const __half2*>(&c);
    const __half2 n = i & 1 ? __hfma2(a, __float2half2_rn(0.0625f), __float2half2_rn(-64.0f)) : __hsub2(a, __float2half2_rn(1024.0f));
    const __half2 v = __hfma2(n, scale, low);
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint32_t at_most_65504(uint32_t v) {
  const __half2 x = __hmin2_nan(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(65504.0f));
  return *reinterpret_cast<const uint32_t*>(&x);
}

// The larger of three; two fp32 values in one register pair, a multiply-add or a sum of both at once.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void halves(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1) kv_tc_kernel(Params p, int* __restrict__ err) {
  using C = Cfg<D>;
  constexpr int NC = C::NC, NM = C::NM;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* c_full = reinterpret_cast<uint64_t*>(smem + C::BARS);    // packed tiles
  uint64_t* c_empty = c_full + NC;
  uint64_t* m_full = c_empty + NC;                                   // dequantized matrices: K, V, K, V, ...
  uint64_t* m_empty = m_full + NM;
  uint64_t* q_full = m_empty + NM;                                   // per group from here on
  uint64_t* s_full = q_full + 2;                                     // per group and half of a tile
  uint64_t* p_full = s_full + 4;
  uint64_t* o_done = p_full + 4;                                     // P V of a half tile is done
  uint64_t* o_last = o_done + 2;                                     // the item's last P V is
  uint64_t* o_free = o_last + 2;                                     // the item's O has been read
  uint64_t* drain = o_free + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  long long* sh = reinterpret_cast<long long*>(smem + C::BARS + 384);        // 14 values

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NC; ++i) {
      mbar_init(&c_full[i], 1);
      mbar_init(&c_empty[i], NDEQ);
    }
    for (int i = 0; i < NM; ++i) {
      mbar_init(&m_full[i], NDEQ);
      mbar_init(&m_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&s_full[2 * i + b], 1);
        mbar_init(&p_full[2 * i + b], 4);
      }
      mbar_init(&o_done[i], 1);
      mbar_init(&o_last[i], 1);
      mbar_init(&o_free[i], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  Line<R, kItemCost> line;
  line.init(p, sh, err);                                             // its barriers order the above too
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t s_tm = tmem, o_tm = tmem + 256;                     // S (and P) of group x at + 128 x, O at + D x
  grid_dep_launch();
  Item it;
  bool ok = true;
  auto give_up = [&]() {
    ok = false;
    *abort_flag = 1;
    if (lane == 0) report_device_error(err, DEVERR_TIMEOUT);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_ISSUE));
    if (warp == 0) {
      // ---------------- copies of the packed tiles ----------------
      Copies cp;
      cp.init(p, lane);
      uint32_t n = 0;
      while (ok && line.next(p, it)) {
        long long src = cp.source(p, it, 0, D, err);
        for (int i = 0; i < it.nt; ++i, ++n) {
          const uint32_t st = n % NC;
          const long long next = cp.source(p, it, i + 1, D, err);
          if (!mbar_wait_bounded(&c_empty[st], (n / NC & 1u) ^ 1u, abort_flag)) { give_up(); break; }
          cp.issue(p, smem_u32(smem) + C::CODES + st * C::STAGE, &c_full[st], src, D, lane);
          src = next;
        }
      }
      for (uint32_t u = n > NC ? n - NC : 0; u < n; ++u) mbar_wait_bounded(&c_full[u % NC], u / NC & 1u, nullptr);
    } else if (warp == 1) {
      // ---------------- MMA issuer ----------------
      const uint32_t leader = elect_leader();
      constexpr uint32_t IDS = umma_idesc(/*f16*/ 0, false, false, 128, 64), IDO = umma_idesc(0, false, /*B MN-major*/ true, 128, D);
      const uint32_t sb = smem_u32(smem);
      const uint64_t q_desc = umma_sdesc_sw128(sb, 16, 1024), k_desc = umma_sdesc_sw128(sb + C::MATS, 16, 1024);
      const uint64_t v_desc = umma_sdesc_sw128(sb + C::MATS, C::BOX, 1024);
      uint32_t mat = 0, np[4] = {0, 0, 0, 0}, items[2] = {0, 0};     // matrices; waits per group and half; items per group
      bool issued = false;
      // S of half tile j into its half of the group's columns
      auto scores = [&](int x, int j, uint32_t kslot) {
        const uint64_t kd = k_desc + (uint64_t)(kslot * (C::MAT / 16) + (j & 1) * (64 * 128 / 16)), qd = q_desc + (uint64_t)(x * (C::MAT / 16));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_f16_ss(s_tm + 128 * x + 64 * (j & 1), qd + (kk >> 2) * (C::BOX / 16) + 2 * (kk & 3),
                      kd + (kk >> 2) * (C::BOX / 16) + 2 * (kk & 3), IDS, kk > 0, leader);
        commit_by(&s_full[2 * x + (j & 1)], leader);
      };
      while (ok && line.next(p, it)) {
        const int groups = it.rows > 128 ? 2 : 1, nh = 2 * it.nt;    // half tiles
        if (nh == 0) continue;
        // the first tile's scores; K is number mat, V number mat + 1 of the ring's matrices
        if (!mbar_wait_poll(&m_full[mat % NM], mat / NM & 1u, abort_flag)) { give_up(); break; }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (x >= groups) break;
          if (!mbar_wait_poll(&q_full[x], items[x] & 1u, abort_flag) ||
              !mbar_wait_poll(&o_free[x], (items[x] & 1u) ^ 1u, abort_flag)) { give_up(); break; }
          ++items[x];
          tc_fence_after();
          issued = true;
          scores(x, 0, mat % NM);
          scores(x, 1, mat % NM);
        }
        if (!ok) break;
        commit_by(&m_empty[mat % NM], leader);
        // P V of half tile j, then S of half tile j + 2 over that P
        for (int j = 0; ok && j < nh; ++j) {
          const uint32_t vn = mat + 1 + (j & ~1), kn = vn + 1, vslot = vn % NM, kslot = kn % NM;
          if (!(j & 1) && !mbar_wait_poll(&m_full[vslot], vn / NM & 1u, abort_flag)) { give_up(); break; }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (x >= groups) break;
            const int b = 2 * x + (j & 1);
            if (!mbar_wait_poll(&p_full[b], (j & 1 ? np[2 * x + 1] : np[2 * x]) & 1u, abort_flag)) { give_up(); break; }
            if (j & 1) ++np[2 * x + 1]; else ++np[2 * x];
            tc_fence_after();
            const uint64_t vd = v_desc + (uint64_t)(vslot * (C::MAT / 16) + (j & 1) * (64 * 128 / 16));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)                           // 16 keys: 16 rows of 128 bytes
              umma_f16_ts(o_tm + D * x, s_tm + 128 * x + 64 * (j & 1) + 8 * kk, vd + kk * 128, IDO, j > 0 || kk > 0,
                          leader);
            commit_by(&o_done[x], leader);
            if (j == nh - 1) commit_by(&o_last[x], leader);
            if ((j & 1) && x == groups - 1) commit_by(&m_empty[vslot], leader);
            if (j + 2 < nh) {
              if (x == 0 && !(j & 1)) {
                if (!mbar_wait_poll(&m_full[kslot], kn / NM & 1u, abort_flag)) { give_up(); break; }
                tc_fence_after();
              }
              scores(x, j, kslot);
              if ((j & 1) && x == groups - 1) commit_by(&m_empty[kslot], leader);
            }
          }
        }
        mat += 2 * (uint32_t)it.nt;
      }
      if (issued) {
        commit_by(drain, leader);
        mbar_wait_bounded(drain, 0, nullptr);
      }
    }
  } else if (warp < SOFT0) {
    // ---------------- dequantize: a thread holds one half of one key of the tile ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_DEQ));
    constexpr int NW = D / 16;                                       // words of half a row
    const int r = (tid - 32 * DEQ0) & 127, half = (tid - 32 * DEQ0) >> 7, blk = r >> p.pb_log2, at = r & (p.pb - 1);
    const uint32_t off = blk * p.pb * (D + 8) + at * (D / 2) + half * (D / 4), noff = blk * p.pb * (D + 8) + p.pb * D + at * 8;
    const uint32_t sb = smem_u32(smem), sw = r & 7;
    uint32_t n = 0, mat = 0;
    while (ok && line.next(p, it)) {
      for (int i = 0; i < it.nt; ++i, ++n) {
        const uint32_t st = n % NC, base = sb + C::CODES + st * C::STAGE;
        if (!mbar_wait_bounded(&c_full[st], n / NC & 1u, abort_flag)) { give_up(); break; }
        const bool live = (it.tl + i) * TILE + r < it.hi_all;        // past the end anything may lie there
        uint32_t num[2];
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(num[0]), "=r"(num[1]) : "r"(base + noff));
        if (!live) num[0] = num[1] = 0u;
        const float2 kn = __half22float2(*reinterpret_cast<const __half2*>(&num[0]));
        const float2 vn = __half22float2(*reinterpret_cast<const __half2*>(&num[1]));
        const float any = kn.x + kn.y + vn.x + vn.y;                 // finite numbers, or a NaN among them
        if (any != any) { num[0] = 0x7FFF7FFFu; num[1] = 0u; }
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++mat) {
          const uint32_t slot = mat % NM;
          uint32_t w[NW];
#pragma unroll
          for (int c = 0; c < NW; c += 4)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[c]), "=r"(w[c + 1]), "=r"(w[c + 2]), "=r"(w[c + 3])
                         : "r"(base + off + kv * p.pb * (D / 2) + 4 * c));
          if (!mbar_wait_bounded(&m_empty[slot], (mat / NM & 1u) ^ 1u, abort_flag)) { give_up(); break; }
          const uint32_t nn = kv ? num[1] : num[0];
          const __half2 s = __half2half2(__ushort_as_half((unsigned short)nn));
          const __half2 l = __half2half2(__ushort_as_half((unsigned short)(nn >> 16)));
          // 15 * scale + low can round past fp16's largest number: such values are kept at that number
          const bool past = __any_sync(0xffffffffu, fmaf(15.0f, __low2float(s), __low2float(l)) > 65504.0f);
          const uint32_t dst = sb + C::MATS + slot * C::MAT + r * 128;
#pragma unroll
          for (int c = 0; c < NW; ++c) {
            const int cc = half * NW + c;                            // the row's 16-byte piece
            uint4 v = dequant8(w[c], s, l);
            if (past) v = make_uint4(at_most_65504(v.x), at_most_65504(v.y), at_most_65504(v.z), at_most_65504(v.w));
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + (cc >> 3) * C::BOX + (((cc & 7) ^ sw) << 4)), "r"(v.x),
                         "r"(v.y), "r"(v.z), "r"(v.w)
                         : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&m_full[slot]);
            if (kv == 1) mbar_arrive(&c_empty[st]);      // here its words have been read: loads alone may still be on their way
          }
        }
        if (!ok) break;
      }
    }
  } else {
    // ---------------- softmax: a query row per thread, group x ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_SOFT));
    const int x = (warp - SOFT0) >> 2, r = tid - 32 * SOFT0 - 128 * x;          // this group's row
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t st0 = s_tm + 128 * x + lanes, ot = o_tm + D * x + lanes;
    uint32_t ns[2] = {0, 0}, npv = 0, no = 0;                        // waits for S by half tile; half tiles whose P V was asked for; items
    int4 cut = make_int4(0, 0, 0, 0);
    while (ok && line.next(p, it)) {
      if (it.more) cut = make_int4(it.b, it.item, 1 + it.more, 0);
      if (x == 1 && it.rows <= 128) continue;
      const int rr = it.rt * R + 128 * x + r, tk = rr / p.G, hq = it.h * p.G + rr - tk * p.G;
      const bool row_ok = 128 * x + r < it.rows;
      const int pos0 = it.sq.len - it.sq.nq;
      const long long lo_l = p.window > 0 ? (long long)pos0 + tk - p.window + 1 : 0;
      const int lo = lo_l > 0 ? (lo_l < 0x7FFFFFFF ? (int)lo_l : 0x7FFFFFFF) : 0;
      const int hi = !row_ok ? -1 : (p.causal ? min(it.sq.len - 1, pos0 + tk) : it.sq.len - 1);
      // tiles in which every row of the group sees every key need no mask
      const int g0 = (it.rt * R + 128 * x) / p.G, g1 = (it.rt * R + min(128 * x + 127, it.rows - 1)) / p.G;
      const int hi_min = p.causal ? min(it.sq.len, max(0, pos0 + g0 + 1)) : it.sq.len;
      const long long lo1 = p.window > 0 ? (long long)pos0 + g1 - p.window + 1 : 0;
      const int lo_max = lo1 > 0 ? (int)(lo1 < it.sq.len ? lo1 : it.sq.len) : 0;
      // ---- the row into shared memory as fp16, scaled by a power of two
      float rowc;
      {
        const uint16_t* qp = reinterpret_cast<const uint16_t*>(p.Q) + (it.sq.tok0 + tk) * p.ldq + (long long)hq * D;
        float mx = 0.0f;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (row_ok) w = *reinterpret_cast<const uint4*>(qp + 8 * c);
          float v[8];
          if (p.q_f16) unpack8<F16>(&w, v); else unpack8<BF16>(&w, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(v[k]));
        }
        const int e = row_exponent(mx);
        const float f = pow2(e);
        // not 0, which would make a NaN of the -infinity of an unseen key; that low, scores round to 0 anyway
        rowc = fmaxf(p.scale_log2 * pow2(-e), 1.17549435e-38f);
        const uint32_t dst = smem_u32(smem) + x * C::MAT + r * 128;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (row_ok) w = *reinterpret_cast<const uint4*>(qp + 8 * c);
          float v[8];
          if (p.q_f16) unpack8<F16>(&w, v); else unpack8<BF16>(&w, v);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + (c >> 3) * C::BOX + (((c & 7) ^ (r & 7)) << 4)),
                       "r"(pack_half2(v[0] * f, v[4] * f)), "r"(pack_half2(v[1] * f, v[5] * f)), "r"(pack_half2(v[2] * f, v[6] * f)),
                       "r"(pack_half2(v[3] * f, v[7] * f))
                       : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && it.nt > 0) mbar_arrive(&q_full[x]);
      }
      float mrc = 0.0f, thr = -CUDART_INF_F, l = 0.0f;               // maximum in log2 units (0: none yet), its limit, the sum
      for (int j = 0; j < 2 * it.nt; ++j) {
        const int b = j & 1;
        if (!mbar_wait_bounded(&s_full[2 * x + b], (b ? ns[1] : ns[0]) & 1u, abort_flag)) { give_up(); break; }
        if (b) ++ns[1]; else ++ns[0];
        tc_fence_after();
        const uint32_t st = st0 + 64 * b;
        const int key0 = it.tl * TILE + 64 * j;
        const bool masked = key0 < lo_max || key0 + 64 > hi_min;
        const int u_lo = lo - key0, u_hi = hi - key0;                // columns the row sees
        // One pass computes the probabilities from the maximum so far and this tile's maximum. Only
        // where that is more than 2^kSlack above (an item's first tile, seldom later) the row moves
        // its maximum and the pass is done again.
        uint32_t pw[32];
        float s0, s1;
#pragma unroll 1
        for (;;) {
          const float sh = kShift - mrc;
          const uint64_t b2 = pair(sh, sh), rowc2 = pair(rowc, rowc);
          uint64_t sum[2] = {0, 0};
          float m4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
          uint32_t s[2][CH];
          tmem_ld32(st, s[0]);
#pragma unroll
          for (int c = 0; c < 64; c += CH) {
            uint32_t* v = s[c / CH & 1];
            tmem_ld_wait<CH>(v);
            if (c + CH < 64) tmem_ld32(st + c + CH, s[1 - (c / CH & 1)]);
            if (masked) {
              const int a = u_lo - c, z = u_hi - c;
              constexpr uint32_t all = 0xFFFFFFFFu >> (32 - CH);
              const uint32_t see = (a >= CH || z < 0) ? 0u : (a > 0 ? all << a : all) & (z < CH - 1 ? all >> (CH - 1 - z) : all);
#pragma unroll
              for (int k = 0; k < CH; ++k)
                if (!(see >> k & 1u)) v[k] = 0xFF800000u;            // -infinity
            }
#pragma unroll
            for (int k = 0; k < CH; k += 2) {
              m4[k / 2 & 3] = max3(m4[k / 2 & 3], __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
              float e0, e1;
              halves(fma2(pair(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), rowc2, b2), e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              sum[k / 2 & 1] = add2(sum[k / 2 & 1], pair(e0, e1));
              pw[(c + k) / 2] = pack_half2(e0, e1);
            }
          }
          halves(add2(sum[0], sum[1]), s0, s1);
          const float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * rowc;
          const bool over = mx > thr;
          if (!__any_sync(0xffffffffu, over)) break;
          float f = 1.0f;
          if (over) {
            f = thr == -CUDART_INF_F ? 0.0f : ex2(mrc - mx);
            mrc = mx;
            thr = mx + kSlack;
            l *= f;
          }
          if (j > 0) {
            // O is this group's own; the P V before has to be done (the one before that is: this S was
            // issued after it, so the barrier is at this phase or past it)
            if (!mbar_wait_bounded(&o_done[x], (npv - 1) & 1u, abort_flag)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 8) {
              uint32_t o[8];
              tmem_ld8(ot + c, o);
              tmem_ld_wait<8>(o);
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st8(ot + c, o);
            }
          }
        }
        if (!ok) { give_up(); break; }
        l += s0 + s1;
        tmem_st32(st, pw);                       // over scores that have been read
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * x + b]);
        ++npv;
      }
      if (!ok) break;
      // ---- the item's output
      if (it.nt > 0) {
        if (!mbar_wait_bounded(&o_last[x], no & 1u, abort_flag)) { give_up(); break; }
        ++no;
        tc_fence_after();
      }
      const long long at = (it.sq.tok0 + tk) * p.ldo + (long long)hq * D;
      float* out = p.part + (2LL * blockIdx.x + (it.lead ? 0 : 1)) * C::PART;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        if (it.nt > 0) {
          tmem_ld8(ot + c, o);
          tmem_ld8(ot + c + 8, o + 8);
          tmem_ld_wait<16>(o);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          if (!row_ok) break;
          const int e = (k & ~7) + (k >> 2 & 1);                     // column j of eight lies at 2 (j mod 4) + j / 4
          float4 w = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 2]), __uint_as_float(o[e + 4]), __uint_as_float(o[e + 6]));
          if (l == 0.0f) w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);    // no key seen: O may never have been written
          const int col = c + k;
          if (it.whole) store_out(p, at + col, make_float4(w.x * inv, w.y * inv, w.z * inv, w.w * inv));
          else *reinterpret_cast<float4*>(out + (128 * x + r) * D + col) = w;
        }
      }
      if (row_ok) {
        if (it.whole) {
          if (p.lse) p.lse[(it.sq.tok0 + tk) * p.Hq + hq] = l == 0.0f ? -CUDART_INF_F : (mrc - kShift + log2f(l)) * 0.6931471805599453f;
        } else {
          out[R * D + 128 * x + r] = l == 0.0f ? -CUDART_INF_F : mrc - kShift;
          out[R * D + R + 128 * x + r] = l;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && it.nt > 0) mbar_arrive(&o_free[x]);
    }
    if (tid == 32 * SOFT0) p.cut[blockIdx.x] = cut;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace tc
}  // namespace kva

size_t kv_attention_tc_workspace_bytes(int D) {
  using namespace kva;
  const size_t part = D == 64 ? tc::Cfg<64>::PART : tc::Cfg<128>::PART, ctas = (size_t)sm_count();
  return round256(16 * ctas) + ctas * 2 * part * 4;
}

template <int D>
static gptq_status tc_launch(kva::Params p, void* ws, cudaStream_t s) {
  using namespace kva;
  using C = tc::Cfg<D>;
  static PerDevice done;
  if (gptq_status st = allow_smem(done, tc::kv_tc_kernel<D>, C::SMEM, "kv_tc_kernel")) return st;
  const unsigned ctas = (unsigned)sm_count();
  p.cut = reinterpret_cast<int4*>(ws);
  p.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + round256(16 * (size_t)ctas));
  tc::kv_tc_kernel<D><<<ctas, tc::THREADS, C::SMEM, s>>>(p, device_error_word());
  count_launch();
  if (gptq_status st = check_launch("kv_tc_kernel")) return st;
  launch_pdl(kv_join_kernel<D, tc::R>, dim3(ctas, 8), dim3(JOIN_WARPS * 32), 0, s, p);
  count_launch();
  return check_launch("kv_join_kernel");
}

gptq_status kv_attention_tc_launch(const kva::Params& p, int D, void* ws, cudaStream_t s) {
  return D == 64 ? tc_launch<64>(p, ws, s) : tc_launch<128>(p, ws, s);
}

}  // namespace gptq
