// A packed projection of many tokens with what follows it (gptq_linear without adapters):
//
//   Y[t][r] = act(x_scale[t] * sum_g scale[r][g] * sum_{j in g} X[t][j] (code[r][j] - zero[r][g]) + bias[r]) * mul[t][r]
//             + residual[t][r]
//
// Tiles of 128 rows by 256 tokens on the 5th-generation tensor cores, one persistent CTA an SM. X comes by
// TMA, bf16 or e4m3; W_hat's integers are unpacked from the codes into the other operand in shared
// memory, as numbers of X's type, exactly: bf16 holds (code - zero) * 2^-6, and e4m3, whose numbers below 2^-5 are
// whole multiples of 2^-9 in the order of their bits, holds (code - zero) * 2^-9 for up to 4 bits as the
// magnitude itself with a sign bit. The factors go into the scale. Products are exact in fp32.
// The sum of a group (or of 128 columns of it) leaves tensor memory through the epilogue warps, which add it times
// the row's scale, a value per lane, in fp32.
//
//   warp 0       TMA producer of X: slabs of 128 bytes of a token's row (64 columns of bf16, 128 of e4m3)
//   warp 1       MMA issuer: four MMAs of M 128, N 256 a slab, an accumulator per unit, two in turn (all of
//                tensor memory, so W_hat's operand is in shared memory)
//   warp 2       TMA producer of the packed codes
//   warp 3       the scales of the next units
//   warps 4-11   unpack: a lane takes 32 columns of a row at a time
//   warps 12-27  epilogue: a warp has 32 rows (its tensor-memory lanes) and 64 tokens
//
// A unit of 128 columns is 1024 cycles of MMAs in bf16 and 512 in e4m3; the epilogue's 512 paired fp32 multiply-adds
// share the schedulers with the unpacking (about 11 instructions per 8 codes). Sixteen epilogue warps of 64 sums a
// thread hide the loads from tensor memory; eight of 128 would take the registers of twice as many.
//
// Measured: 8192 x 8192, 4096 tokens 345 us in bf16 (1.59 PFLOP/s, 92 % of the library's sustained rate), 320 in e4m3 (1.72); 28672 x
// 8192, 2500 tokens in e4m3 663 us (1.77 PFLOP/s). Bound: the issue slots that unpacking and epilogue share (e4m3 without
// the unpacking: 225 us), power beyond that.
#include <algorithm>
#include <type_traits>

#include "packed.cuh"
#include "ring.h"

namespace gptq {
namespace ltl {

using namespace adp;

constexpr int NTOK = 256, ND = 2;
constexpr int UNPACK0 = 4, NUNPACK = 8, EPI0 = 12, NEPI = 16, THREADS = (EPI0 + NEPI) * 32;
constexpr int SCALES = 4, S_STAGES = 2;                  // units whose scales are staged together, and how often
constexpr int COLS = 64;                                 // tokens of an epilogue warp
// 4 warps of 40 + 8 of 40 + 16 of 96 = 2016 = 28 warps of the 72 that the block has at launch
constexpr int REG_ISSUE = 40, REG_UNPACK = 40, REG_EPI = 96;
constexpr int A_SLAB = BM * 128, X_SLAB = NTOK * 128;

struct Params {
  const uint32_t* qweight;
  const float* scales;
  const float* zeros;
  const float* x_scale;
  const float* bias;
  const void* mul;
  const void* residual;
  void* Y;
  long long ldy, ldm, ldr;
  int m, d, T, gs, G, wpr, unit, act, y_bf16, codes_tma;
  uint32_t gs32_mul;           // ceil(2^32 / (gs / 32)), 0 when gs is 32
  int d_pad;                   // d in whole blocks
  int mt, nt, group;           // row tiles, token tiles, token tiles that are walked together
};

// The unpacking warps form sets that take slabs in turn, so that one set's waits pass beside another's work: four, where
// shared memory has room for as many slabs and their codes (8192 x 8192, 4096 tokens in bf16: 345 us, with two 375; at 4 bits
// in e4m3, where it has room for three blocks of codes, two: 317 to 324, with four 320).
template <int BITS, bool BYTES>
struct Cfg {
  static constexpr int KC = BYTES ? 128 : 64;              // columns of a slab
  static constexpr int ROW_BYTES = 16 * BITS;              // packed codes of a row in one block of 128 columns
  static constexpr int C_BYTES = (BM * ROW_BYTES + 1023) / 1024 * 1024;
  static constexpr int STAGES = BITS == 8 ? 3 : 4, CODE_STAGES = BITS == 8 ? 2 : (BITS == 4 ? 3 : 4);
  static constexpr int SETS = BITS == 8 || (BYTES && BITS == 4) ? 2 : 4;
  static constexpr int S_BYTES = S_STAGES * SCALES * BM * 4;                   // scales, and zeros as many
  static constexpr int SMEM = STAGES * (A_SLAB + X_SLAB) + CODE_STAGES * C_BYTES + 2 * S_BYTES + 1024 + 256;
  static_assert(SMEM <= 232448, "more than an SM has");
  // Barriers of the slabs that are free again and of the blocks that have landed, for sets that skip the others' (ring.h). A
  // row's last block counts as whole, so that a set's step is the same from tile to tile.
  static constexpr int BLOCK_STEP = SETS * KC > KB ? SETS * KC / KB : 1;
  static constexpr int EMPTIES = barriers_for(STAGES, SETS), C_FULLS = barriers_for(CODE_STAGES, BLOCK_STEP);
  static constexpr int BARRIERS = STAGES + EMPTIES + C_FULLS + CODE_STAGES + 2 * ND + 4 * S_STAGES + 1;
  static_assert(8 * BARRIERS + 8 <= 256, "more barriers than have room");
};

__device__ __forceinline__ void umma(bool bytes, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate,
                                     uint32_t leader) {
  if (bytes)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}

// 32 codes (BITS words) as bytes in the columns' order.
template <int BITS>
__device__ __forceinline__ void spread32(const uint32_t* w, uint32_t (&o)[8]) {
  if constexpr (BITS == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t e = w[j] & 0x0F0F0F0Fu, d = (w[j] >> 4) & 0x0F0F0F0Fu;
      o[2 * j] = prmt(e, d, 0x5140u);
      o[2 * j + 1] = prmt(e, d, 0x7362u);
    }
  } else if constexpr (BITS == 2) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = (w[j] >> (2 * k)) & 0x03030303u;
      const uint32_t a = prmt(c[0], c[1], 0x5140u), b = prmt(c[2], c[3], 0x5140u);
      const uint32_t e = prmt(c[0], c[1], 0x7362u), f = prmt(c[2], c[3], 0x7362u);
      o[4 * j] = prmt(a, b, 0x5410u);
      o[4 * j + 1] = prmt(a, b, 0x7632u);
      o[4 * j + 2] = prmt(e, f, 0x5410u);
      o[4 * j + 3] = prmt(e, f, 0x7632u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {                          // 12 bits from bit 12 i on
      const int b = 12 * i, k = b >> 5, sh = b & 31;
      const uint32_t s = k < 2 ? __funnelshift_r(w[k], w[k + 1], sh) : w[2] >> sh;
      o[i] = (s & 0x7u) | ((s << 5) & 0x700u) | ((s << 10) & 0x70000u) | ((s << 15) & 0x7000000u);
    }
  }
}
// Four bytes of codes c to e4m3 bits of (c - z) * 2^-9; kz = 0x80808080 - z in every byte, so that a byte of c + kz has
// its top bit where c >= z.
__device__ __forceinline__ uint32_t minus_zero(uint32_t c, uint32_t kz) {
  return __vabsdiffu4(c, 0x80808080u - kz) | (~(c + kz) & 0x80808080u);
}

// BITS words of 32 columns (quarter q of a block) of row r of a stage of packed codes.
template <int BITS>
__device__ __forceinline__ void lds_quarter(uint32_t stage, int r, int q, uint32_t* w) {
  if constexpr (BITS == 4) {
    lds_piece<4>(stage, r, q, w);
  } else if constexpr (BITS == 8) {
    lds_piece<8>(stage, r, 2 * q, w);
    lds_piece<8>(stage, r, 2 * q + 1, w + 4);
  } else if constexpr (BITS == 2) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                 : "=r"(w[0]), "=r"(w[1])
                 : "r"(stage + r * 32 + (((q >> 1) ^ ((r >> 2) & 1)) * 16 + (q & 1) * 8)));
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[i]) : "r"(stage + r * 48 + 12 * q + 4 * i));
  }
}
// A block of codes of 128 rows from word `w0` of each on, as TMA would lay it out; what lies outside is 0.
template <int BITS>
__device__ __forceinline__ void copy_codes(const Params& p, uint32_t stage, int r0, int w0, int lane) {
  constexpr int WORDS = 4 * BITS;
  for (int x = lane; x < BM * WORDS; x += 32) {
    const int r = x / WORDS, w = x - r * WORDS, i = w / 4;
    const int at = BITS == 8 ? i ^ (r & 7) : BITS == 4 ? i ^ ((r >> 1) & 3) : BITS == 2 ? i ^ ((r >> 2) & 1) : i;
    const uint32_t v = r0 + r < p.m && w0 + w < p.wpr ? __ldg(p.qweight + (long long)(r0 + r) * p.wpr + w0 + w) : 0u;
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(stage + r * (16 * BITS) + at * 16 + (w & 3) * 4), "r"(v) : "memory");
  }
}
__device__ __forceinline__ void sts16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Tile i: token tiles in groups that are walked before the next row tile, so that the CTAs at work share
// rows of codes and X's tiles in L2.
__device__ __forceinline__ void tile_of(const Params& p, int i, int& rt, int& tt) {
  const int per = p.group * p.mt, g = i / per, in = i - g * per, n = min(p.group, p.nt - g * p.group);
  rt = in / n;
  tt = g * p.group + (in - rt * n);
}

// What follows the product, in steps over a thread's 64 sums of one row, each step one straight run of code: as a loop over
// the sums the registers would have to move, and with the choices inside, the code of all of them would be read for
// every tile. n: tokens of the 64 that there are (0 in a lane without a row).
// in_turn: what is computed from these sums comes after what was before it, so that the registers of few are in use at once.
template <int N>
__device__ __forceinline__ void in_turn(uint64_t* run) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) asm volatile("" : "+l"(run[i]));
}
template <typename E, bool MUL>
__device__ __forceinline__ void take_in(const void* p, long long at, long long ld, int n, uint64_t (&run)[COLS / 2]) {
  const typename E::T* x = reinterpret_cast<const typename E::T*>(p) + at;
  constexpr int AT = 8;                                    // values on their way together
#pragma unroll
  for (int c = 0; c < COLS; c += AT) {
    typename E::T v[AT];
#pragma unroll
    for (int i = 0; i < AT; ++i, x += ld) v[i] = c + i < n ? *x : typename E::T(0.0f);
#pragma unroll
    for (int i = 0; i < AT; i += 2) {
      const float v0 = (float)v[i], v1 = (float)v[i + 1];
      uint64_t& r = run[(c + i) / 2];
      r = MUL ? pack2(half2f(r, 0) * v0, half2f(r, 1) * v1) : pack2(half2f(r, 0) + v0, half2f(r, 1) + v1);
    }
    in_turn<AT>(&run[c / 2]);
    asm volatile("" : "+l"(x));
  }
}
template <typename E>
__device__ __forceinline__ void put_out(void* p, long long at, long long ld, int n, const uint64_t (&run)[COLS / 2]) {
  typename E::T* y = reinterpret_cast<typename E::T*>(p) + at;
#pragma unroll
  for (int c = 0; c < COLS; ++c, y += ld) {
    if (c < n) *y = (typename E::T)half2f(run[c / 2], c & 1);
    if (c % 4 == 3) asm volatile("" : "+l"(y));
  }
}
__device__ __forceinline__ void finish(const Params& p, int t, int row, bool live, uint64_t (&run)[COLS / 2]) {
  const int n = live ? min(COLS, p.T - t) : 0;
  const float bias = p.bias && live ? __ldg(p.bias + row) : 0.0f;
  if (p.x_scale) {
    int last = p.T - 1;
#pragma unroll
    for (int c = 0; c < COLS; c += 16) {
      float sx[16];
      asm volatile("" : "+r"(last));
#pragma unroll
      for (int i = 0; i < 16; ++i) sx[i] = __ldg(p.x_scale + min(t + c + i, last));
#pragma unroll
      for (int i = 0; i < 16; i += 2) run[(c + i) / 2] = fma2(run[(c + i) / 2], pack2(sx[i], sx[i + 1]), pack2(bias, bias));
      in_turn<16>(&run[c / 2]);
    }
  } else if (p.bias) {
#pragma unroll
    for (int c = 0; c < COLS; c += 2) run[c / 2] = add2(run[c / 2], pack2(bias, bias));
  }
  auto all = [&](int act) {
#pragma unroll
    for (int c = 0; c < COLS; c += 4) {
      in_turn<4>(&run[c / 2]);
#pragma unroll
      for (int i = c / 2; i < c / 2 + 2; ++i) run[i] = pack2(activate(half2f(run[i], 0), act), activate(half2f(run[i], 1), act));
      in_turn<4>(&run[c / 2]);
    }
  };
  if (p.act == GPTQ_ACT_SILU) all(GPTQ_ACT_SILU);
  else if (p.act == GPTQ_ACT_RELU) all(GPTQ_ACT_RELU);
  else if (p.act == GPTQ_ACT_GELU) {
    // too long to be repeated 64 times: the sums go around, eight at a time
#pragma unroll 1
    for (int k = 0; k < COLS / 8; ++k) {
      uint64_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = pack2(activate(half2f(run[i], 0), GPTQ_ACT_GELU), activate(half2f(run[i], 1), GPTQ_ACT_GELU));
#pragma unroll
      for (int i = 0; i < COLS / 2 - 4; ++i) run[i] = run[i + 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) run[COLS / 2 - 4 + i] = v[i];
    }
  }
  else if (p.act == GPTQ_ACT_GELU_TANH) all(GPTQ_ACT_GELU_TANH);
  if (p.mul) {
    if (p.y_bf16) take_in<BF16, true>(p.mul, t * p.ldm + row, p.ldm, n, run);
    else take_in<F32, true>(p.mul, t * p.ldm + row, p.ldm, n, run);
  }
  if (p.residual) {
    if (p.y_bf16) take_in<BF16, false>(p.residual, t * p.ldr + row, p.ldr, n, run);
    else take_in<F32, false>(p.residual, t * p.ldr + row, p.ldr, n, run);
  }
  if (p.y_bf16) put_out<BF16>(p.Y, t * p.ldy + row, p.ldy, n, run);
  else put_out<F32>(p.Y, t * p.ldy + row, p.ldy, n, run);
}

template <int BITS, bool BYTES>
__global__ void __launch_bounds__(THREADS, 1)
linear_tiles_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_c, Params p, int* __restrict__ err) {
  using C = Cfg<BITS, BYTES>;
  constexpr int KC = C::KC, KSTEP = KC / 4;                // columns of a slab, of an MMA
  constexpr int STAGES = C::STAGES, CODE_STAGES = C::CODE_STAGES, SETS = C::SETS, SET = NUNPACK / SETS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* xs = smem + STAGES * A_SLAB;
  uint8_t* codes = xs + STAGES * X_SLAB;
  float* scales = reinterpret_cast<float*>(codes + CODE_STAGES * C::C_BYTES);
  uint32_t* zeros = reinterpret_cast<uint32_t*>(scales + C::S_BYTES / 4);      // in the form that the unpacking takes
  uint64_t* full = reinterpret_cast<uint64_t*>(zeros + C::S_BYTES / 4);
  uint64_t* empty = full + STAGES;
  uint64_t* c_full = empty + C::EMPTIES;
  uint64_t* c_empty = c_full + C::C_FULLS;
  uint64_t* d_full = c_empty + CODE_STAGES;
  uint64_t* d_empty = d_full + ND;
  uint64_t* s_full = d_empty + ND;
  uint64_t* s_empty = s_full + S_STAGES;
  uint64_t* z_full = s_empty + S_STAGES;
  uint64_t* z_empty = z_full + S_STAGES;
  uint64_t* drain = z_empty + S_STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int b = 0; b < STAGES; ++b) mbar_init(&full[b], SET + 1);
    for (int b = 0; b < C::EMPTIES; ++b) mbar_init(&empty[b], 1);
    for (int b = 0; b < C::C_FULLS; ++b) mbar_init(&c_full[b], 1);
    for (int b = 0; b < CODE_STAGES; ++b) mbar_init(&c_empty[b], SET * (KB / KC));
    for (int b = 0; b < ND; ++b) {
      mbar_init(&d_full[b], 1);
      mbar_init(&d_empty[b], NEPI);
    }
    for (int b = 0; b < S_STAGES; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_empty[b], NEPI);
      mbar_init(&z_full[b], 1);
      mbar_init(&z_empty[b], NUNPACK);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_c);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int ntiles = p.mt * p.nt, step = (int)gridDim.x;
  // Slab n's place is free: the MMAs on slab n - STAGES are done, the use of its barrier before u (none, and a new barrier's
  // parity, for the first slabs).
  auto slab_free = [&](uint32_t n) -> bool {
    const uint32_t u = n + (C::EMPTIES - STAGES);
    return mbar_wait_bounded(&empty[u % C::EMPTIES], ((u / C::EMPTIES) & 1u) ^ 1u, abort_flag);
  };
  const bool half = p.d_pad - p.d >= KC;                   // a row's last block has an empty half, a slab of nothing

  if (warp < UNPACK0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_ISSUE));
    if (warp == 0) {
      // ---------------- TMA producer of X ----------------
      uint32_t n = 0;
      bool ok = true;
      for (int tile = (int)blockIdx.x; ok && tile < ntiles; tile += step) {
        int rt, tt;
        tile_of(p, tile, rt, tt);
        for (int k = 0; k < p.d; k += KC, ++n) {
          const uint32_t i = n % STAGES;
          if (!slab_free(n)) { ok = false; break; }
          if (lane == 0) {
            mbar_arrive_expect_tx(&full[i], X_SLAB);
            tma_load_2d(xs + i * X_SLAB, &map_x, &full[i], k, tt * NTOK);
          }
        }
        if (half && ok) {
          if (!slab_free(n)) { ok = false; break; }
          if (lane == 0) mbar_arrive(&full[n % STAGES]);
          ++n;
        }
      }
      if (!ok) { *abort_flag = 1; if (lane == 0) report_device_error(err, DEVERR_TIMEOUT); }
      // copies still in flight when something gave up: their barriers' other arrivals may never come then
      for (uint32_t u = n > STAGES ? n - STAGES : 0; u < n; ++u)
        mbar_wait_bounded(&full[u % STAGES], (u / STAGES) & 1u, nullptr, ok ? kWaitLimitNs : 1000000ull);
    } else if (warp == 1) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t IDESC = umma_idesc(BYTES ? 0 : 1, false, false, BM, NTOK);
      uint32_t n = 0, unit_no = 0;
      bool ok = true;
      const uint32_t leader = elect_leader();
      const uint64_t a0 = umma_sdesc_sw128(smem_u32(smem), 16, 1024), b0 = umma_sdesc_sw128(smem_u32(xs), 16, 1024);
      // The operands in shared memory need no fence behind their barrier's wait, only an accumulator that the epilogue's
      // loads have left: a fence makes the MMAs behind it wait for the ones before.
      auto accumulator = [&]() -> bool {
        if (!mbar_wait_poll(&d_empty[unit_no % ND], ((unit_no / ND) & 1u) ^ 1u, abort_flag)) return false;
        tc_fence_after();
        return true;
      };
      for (int tile = (int)blockIdx.x; ok && tile < ntiles; tile += step) {
        if (p.unit >= KC) {
          const int per = p.unit / KC;                     // slabs of a unit
          int in = 0;                                      // slabs of the present one so far
          for (int k0 = 0; k0 < p.d; k0 += KC, ++n) {
            const uint32_t i = n % STAGES, dt = tmem + (unit_no % ND) * NTOK;
            const uint64_t ad = a0 + (uint64_t)(i * (A_SLAB / 16)), bd = b0 + (uint64_t)(i * (X_SLAB / 16));
            if (in == 0 && !accumulator()) { ok = false; break; }
            if (!mbar_wait_poll(&full[i], (n / STAGES) & 1u, abort_flag)) { ok = false; break; }
            umma(BYTES, dt, ad, bd, IDESC, in != 0, leader);
            if (k0 + KC <= p.d) {
#pragma unroll
              for (int kk = 1; kk < 4; ++kk) umma(BYTES, dt, ad + 2 * kk, bd + 2 * kk, IDESC, 1, leader);
            } else {
              for (int kk = 1; k0 + kk * KSTEP < p.d; ++kk) umma(BYTES, dt, ad + 2 * kk, bd + 2 * kk, IDESC, 1, leader);
            }
            umma_commit_by(&empty[n % C::EMPTIES], leader);
            if (++in == per || k0 + KC >= p.d) {
              umma_commit_by(&d_full[unit_no % ND], leader);
              ++unit_no;
              in = 0;
            }
          }
        } else {                                           // several units in a slab
          for (int k0 = 0; ok && k0 < p.d; k0 += KC, ++n) {
            const uint32_t i = n % STAGES;
            const uint64_t ad = a0 + (uint64_t)(i * (A_SLAB / 16)), bd = b0 + (uint64_t)(i * (X_SLAB / 16));
            if (!mbar_wait_poll(&full[i], (n / STAGES) & 1u, abort_flag)) { ok = false; break; }
            for (int kk = 0; kk < 4 && k0 + kk * KSTEP < p.d; ++kk) {
              const bool begin = ((kk * KSTEP) & (p.unit - 1)) == 0;
              if (begin && !accumulator()) { ok = false; break; }
              umma(BYTES, tmem + (unit_no % ND) * NTOK, ad + 2 * kk, bd + 2 * kk, IDESC, !begin, leader);
              if ((((kk + 1) * KSTEP) & (p.unit - 1)) == 0) {
                umma_commit_by(&d_full[unit_no % ND], leader);
                ++unit_no;
              }
            }
            if (ok) umma_commit_by(&empty[n % C::EMPTIES], leader);
          }
        }
        if (half && ok) {
          if (!mbar_wait_poll(&full[n % STAGES], (n / STAGES) & 1u, abort_flag)) { ok = false; break; }
          umma_commit_by(&empty[n % C::EMPTIES], leader);
          ++n;
        }
      }
      if (!ok) { *abort_flag = 1; if (lane == 0) report_device_error(err, DEVERR_TIMEOUT); }
      umma_commit_by(drain, leader);
      mbar_wait_bounded(drain, 0, nullptr);
    } else if (warp == 2) {
      // ---------------- producer of the packed codes: by TMA, or word by word where it cannot take the rows ----------------
      uint32_t n = 0;
      bool ok = true;
      for (int tile = (int)blockIdx.x; ok && tile < ntiles; tile += step) {
        int rt, tt;
        tile_of(p, tile, rt, tt);
        for (int k = 0; k < p.d; k += KB, ++n) {
          const uint32_t i = n % CODE_STAGES;
          if (!mbar_wait_bounded(&c_empty[i], ((n / CODE_STAGES) & 1u) ^ 1u, abort_flag)) { ok = false; break; }
          if (!p.codes_tma) {
            copy_codes<BITS>(p, smem_u32(codes) + i * C::C_BYTES, rt * BM, k / 32 * BITS, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_full[n % C::C_FULLS]);
          } else if (lane == 0) {
            mbar_arrive_expect_tx(&c_full[n % C::C_FULLS], BM * C::ROW_BYTES);
            tma_load_2d(codes + i * C::C_BYTES, &map_c, &c_full[n % C::C_FULLS], k / KB * C::ROW_BYTES, rt * BM);
          }
        }
      }
      if (!ok) { *abort_flag = 1; if (lane == 0) report_device_error(err, DEVERR_TIMEOUT); }
      for (uint32_t u = n > CODE_STAGES ? n - CODE_STAGES : 0; u < n; ++u) mbar_wait_bounded(&c_full[u % C::C_FULLS], (u / C::C_FULLS) & 1u, nullptr);
    } else if (warp == 3) {
      // ---------------- the scales and zeros of the next units, by row ----------------
      uint32_t n = 0;
      bool ok = true;
      // four groups in a row by one load, where a batch is four groups
      const bool by4 = p.gs == p.unit && (p.G & 3) == 0 && ((reinterpret_cast<uintptr_t>(p.scales) | reinterpret_cast<uintptr_t>(p.zeros)) & 15) == 0;
      auto to_zero = [](float z) -> uint32_t { return BYTES ? 0x80808080u - (uint32_t)(int)z * 0x01010101u : neg_zero(z); };
      for (int tile = (int)blockIdx.x; ok && tile < ntiles; tile += step) {
        int rt, tt;
        tile_of(p, tile, rt, tt);
        for (int k = 0; ok && k < p.d; k += SCALES * p.unit, ++n) {
          const uint32_t i = n % S_STAGES, par = ((n / S_STAGES) & 1u) ^ 1u;
          float* sc = scales + i * SCALES * BM + lane;
          uint32_t* ze = zeros + i * SCALES * BM + lane;
#pragma unroll 1
          for (int what = 0; what < 2; ++what) {           // the zeros, which are needed first, then the scales
            const float* from = what ? p.scales : p.zeros;
            if (by4) {
              float4 v[BM / 32];
#pragma unroll
              for (int j = 0; j < BM / 32; ++j)
                v[j] = __ldg(reinterpret_cast<const float4*>(from + (long long)min(rt * BM + 32 * j + lane, p.m - 1) * p.G + k / p.unit));
              if (!mbar_wait_bounded(what ? &s_empty[i] : &z_empty[i], par, abort_flag)) { ok = false; break; }
#pragma unroll
              for (int j = 0; j < BM / 32; ++j) {
                const float g[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  if (what) sc[u * BM + 32 * j] = g[u] * (BYTES ? 512.0f : 64.0f);
                  else ze[u * BM + 32 * j] = to_zero(g[u]);
                }
              }
            } else {
              if (!mbar_wait_bounded(what ? &s_empty[i] : &z_empty[i], par, abort_flag)) { ok = false; break; }
#pragma unroll 1
              for (int u = 0; u < SCALES; u += 2) {
                float v[2][BM / 32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int c = min(k + (u + h) * p.unit, p.d - 32) / 32, g = p.gs32_mul ? (int)__umulhi((uint32_t)c, p.gs32_mul) : c;
#pragma unroll
                  for (int j = 0; j < BM / 32; ++j) v[h][j] = __ldg(from + (long long)min(rt * BM + 32 * j + lane, p.m - 1) * p.G + g);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int j = 0; j < BM / 32; ++j) {
                    if (what) sc[(u + h) * BM + 32 * j] = v[h][j] * (BYTES ? 512.0f : 64.0f);
                    else ze[(u + h) * BM + 32 * j] = to_zero(v[h][j]);
                  }
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(what ? &s_full[i] : &z_full[i]);
          }
        }
      }
      if (!ok) { *abort_flag = 1; if (lane == 0) report_device_error(err, DEVERR_TIMEOUT); }
    }
  } else if (warp < EPI0) {
    // ---------------- unpack: codes -> registers -> shared memory ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_UNPACK));
    const int u = warp - UNPACK0, set = u / SET, sub = u % SET;
    uint32_t n = 0, cn = 0, zn = 0;                        // slabs, blocks of codes and batches of zeros so far, all sets'
    uint32_t released = 0;                                 // batches of zeros that this warp is done with
    bool ok = true;
    auto fail = [&]() {
      ok = false;
      *abort_flag = 1;
      if (lane == 0) report_device_error(err, DEVERR_TIMEOUT);
    };
    constexpr int ROWS = BM / 32 / SET, QS = KC / 32;      // rows of a lane, quarters of a block in a slab
    const int ush = p.unit == 128 ? 7 : (p.unit == 64 ? 6 : 5);
    // Batches before `upto` are released, each once it was filled: an arrival belongs to the batch, not to the one
    // before it in the same place.
    auto release_to = [&](uint32_t upto) {
      __syncwarp();
      for (; ok && released < upto; ++released) {
        const uint32_t i = released % S_STAGES;
        if (!mbar_wait_bounded(&z_full[i], (released / S_STAGES) & 1u, abort_flag)) { fail(); break; }
        if (lane == 0) mbar_arrive(&z_empty[i]);
      }
    };
    for (int tile = (int)blockIdx.x; ok && tile < ntiles; tile += step) {
      const uint32_t n0 = n;
      // this set's slabs: first, first + SETS, ...
      for (int k = (int)((uint32_t)(set - n0) % SETS) * KC; k < p.d_pad; k += SETS * KC) {
        const uint32_t at = n0 + (uint32_t)(k / KC), i = at % STAGES, cb = cn + (uint32_t)(k / KB), st = cb % CODE_STAGES;
        const uint32_t zb = zn + (uint32_t)(k >> (ush + 2)), zi = zb % S_STAGES;
        release_to(zb);
        if (!ok || !mbar_wait_bounded(&z_full[zi], (zb / S_STAGES) & 1u, abort_flag)) { fail(); break; }
        if (!mbar_wait_bounded(&c_full[cb % C::C_FULLS], (cb / C::C_FULLS) & 1u, abort_flag)) { fail(); break; }
        if (!slab_free(at)) { fail(); break; }
        const uint32_t sc = smem_u32(codes) + st * C::C_BYTES;
        if (k < p.d) {                                     // else an empty half
#pragma unroll
          for (int j = 0; j < ROWS; ++j) {
            const int r = 32 * (ROWS * sub + j) + lane;
            const uint32_t* zr = zeros + (zi * SCALES) * BM + r;
            const uint32_t to = smem_u32(smem) + i * A_SLAB + r * 128, sw = (uint32_t)(r & 7);
#pragma unroll
            for (int q = 0; q < QS; ++q) {
              uint32_t w[BITS];
              const uint32_t z = zr[(((k + 32 * q) >> ush) & (SCALES - 1)) * BM];
              lds_quarter<BITS>(sc, r, (k % KB) / 32 + q, w);
              if constexpr (BYTES) {
                uint32_t o[8];
                spread32<BITS>(w, o);
#pragma unroll
                for (int c = 0; c < 8; ++c) o[c] = minus_zero(o[c], z);
                sts16(to + (((uint32_t)(2 * q) ^ sw) << 4), o[0], o[1], o[2], o[3]);
                sts16(to + (((uint32_t)(2 * q + 1) ^ sw) << 4), o[4], o[5], o[6], o[7]);
              } else {
                uint32_t o[16];
                unpack32<BITS>(w, z, o);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  sts16(to + (((uint32_t)(4 * q + c) ^ sw) << 4), o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
              }
            }
          }
        }
        // for the MMAs that read the slab, and for the next copy of codes: it could overwrite words that a lane's load had
        // not read yet
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[i]);
          mbar_arrive(&c_empty[st]);
        }
      }
      n = n0 + (uint32_t)(p.d_pad / KC);
      cn += (uint32_t)(p.d_pad / KB);
      zn += (uint32_t)((p.d + (SCALES << ush) - 1) >> (ush + 2));
      release_to(zn);
    }
  } else {
    // ---------------- epilogue ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_EPI));
    const int q = warp & 3, h = (warp - EPI0) >> 2;
    const uint32_t td = tmem + ((uint32_t)(32 * q) << 16) + h * COLS;
    uint32_t unit_no = 0;
    bool ok = true;
    uint32_t batch = 0;
    for (int tile = (int)blockIdx.x; ok && tile < ntiles; tile += step) {
      int rt, tt;
      tile_of(p, tile, rt, tt);
      const int row = rt * BM + 32 * q + lane, t0 = tt * NTOK + h * COLS;
      const bool live = row < p.m;
      uint64_t run[COLS / 2];
#pragma unroll
      for (int c = 0; c < COLS / 2; ++c) run[c] = 0ull;
      int su = 0;                                          // units of the present batch of scales so far
      for (int k = 0; k < p.d; k += p.unit) {
        const uint32_t sb = batch % S_STAGES;
        if ((su == 0 && !mbar_wait_bounded(&s_full[sb], (batch / S_STAGES) & 1u, abort_flag)) ||
            !mbar_wait_bounded(&d_full[unit_no % ND], (unit_no / ND) & 1u, abort_flag)) {
          ok = false;
          *abort_flag = 1;
          if (lane == 0) report_device_error(err, DEVERR_TIMEOUT);
          break;
        }
        tc_fence_after();
        const float s = scales[(sb * SCALES + su) * BM + 32 * q + lane];
        const uint64_t ss = pack2(s, s);
        const bool last = ++su == SCALES || k + p.unit >= p.d;
#pragma unroll
        for (int c = 0; c < COLS; c += 16) {
          uint32_t a[16];
          tmem_ld<16>(td + (unit_no % ND) * NTOK + c, a);
          tmem_ld_wait<16>(a);
          if (c == COLS - 16) {                            // all read: the buffers are free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&d_empty[unit_no % ND]);
              if (last) mbar_arrive(&s_empty[sb]);
            }
            ++unit_no;
          }
#pragma unroll
          for (int i = 0; i < 16; i += 2) run[(c + i) / 2] = fma2(pack2u(a[i], a[i + 1]), ss, run[(c + i) / 2]);
        }
        if (last) {
          su = 0;
          ++batch;
        }
      }
      if (!ok) break;
      finish(p, t0, row, live, run);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

bool make_x_map(CUtensorMap* m, const void* base, bool bytes, long long d, long long T, long long ld) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)T};
  cuuint64_t strides[1] = {(cuuint64_t)(ld * (bytes ? 1 : 2))};
  cuuint32_t box[2] = {bytes ? 128u : 64u, NTOK};
  cuuint32_t es[2] = {1, 1};
  return enc(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BITS, bool BYTES>
gptq_status launch(const CUtensorMap& mx, Params p, cudaStream_t s) {
  CUtensorMap mc = mx;
  p.codes_tma = make_code_map(&mc, p.qweight, p.m, (long long)p.wpr * 4, BITS) ? 1 : 0;
  static PerDevice done;
  if (gptq_status st = allow_smem(done, linear_tiles_kernel<BITS, BYTES>, Cfg<BITS, BYTES>::SMEM, "linear_tiles_kernel")) return st;
  const int grid = std::min(p.mt * p.nt, sm_count());
  linear_tiles_kernel<BITS, BYTES><<<grid, THREADS, Cfg<BITS, BYTES>::SMEM, s>>>(mx, mc, p, device_error_word());
  count_launch();
  return check_launch("linear_tiles_kernel");
}

}  // namespace ltl

// X in bf16, or in e4m3 (`bytes`, bits up to 4); x_scale, where there is one, goes with either. The arguments are checked.
gptq_status linear_tiles_launch(const uint32_t* qweight, const float* scales, const float* zeros, long long m, long long d,
                                int bits, int group_size, const void* X, bool bytes, long long T, long long ldx,
                                const float* x_scale, const float* bias, int act, const void* mul, long long ldm,
                                const void* residual, long long ldr, void* Y, int y_dtype, long long ldy,
                                cudaStream_t s) {
  using namespace ltl;
  Params p{};
  p.qweight = qweight; p.scales = scales; p.zeros = zeros; p.x_scale = x_scale; p.bias = bias; p.mul = mul;
  p.residual = residual; p.Y = Y; p.ldy = ldy; p.ldm = ldm; p.ldr = ldr;
  p.m = (int)m; p.d = (int)d; p.T = (int)T;
  p.gs = group_size < 0 ? (int)d : group_size;
  p.G = (int)(d / p.gs);
  p.wpr = (int)(d / 32 * bits);
  p.d_pad = (int)((d + KB - 1) / KB * KB);
  p.unit = p.gs % 128 == 0 ? 128 : (p.gs % 64 == 0 ? 64 : 32);
  p.act = act; p.y_bf16 = y_dtype == GPTQ_BF16;
  const unsigned gs32 = (unsigned)p.gs / 32;
  p.gs32_mul = gs32 == 1 ? 0u : (uint32_t)((0x100000000ULL + gs32 - 1) / gs32);
  const long long mt = (m + BM - 1) / BM, nt = (T + NTOK - 1) / NTOK;
  if (mt * nt > 0x7FFFFFFF - 65536) return set_error(GPTQ_ERR_INVALID_ARG, "too many output tiles");
  p.mt = (int)mt; p.nt = (int)nt; p.group = (int)std::min<long long>(nt, 8);
  CUtensorMap mx;
  if (!make_x_map(&mx, X, bytes, d, T, ldx)) return set_error(GPTQ_ERR_CUDA, "cuTensorMapEncodeTiled failed for X");
  if (bytes) {
    switch (bits) {
      case 2: return launch<2, true>(mx, p, s);
      case 3: return launch<3, true>(mx, p, s);
      default: return launch<4, true>(mx, p, s);
    }
  }
  switch (bits) {
    case 2: return launch<2, false>(mx, p, s);
    case 3: return launch<3, false>(mx, p, s);
    case 4: return launch<4, false>(mx, p, s);
    default: return launch<8, false>(mx, p, s);
  }
}

}  // namespace gptq
