// A packed projection with the low-rank adapters of many requests beside it:
//
//   Y[t] = X[t] W_hat^T + alpha[a] (X[t] A[a]^T) B[a]^T,   a = ids[t]
//   X[t] W_hat[r]^T = sum_g scale[r][g] * sum_{j in g} X[t][j] (code[r][j] - zero[r][g])
//
// adapter_shrink_kernel, adapter_shrink_few_kernel   U[t] = alpha[a] A[a] X[t], alpha[a] in fp32
// adapter_gemm_kernel    the rest, launched behind it without waiting (programmatic launch): it
//                        needs U only after its own sum over d
//
// adapter_gemm_kernel computes a tile of 128 rows of W by N tokens on the 5th-generation tensor
// cores with W_hat's integers as the A operand IN TENSOR MEMORY: the packed words come by TMA into a
// ring in shared memory (rows that TMA cannot take, from global memory); 16 warps, eight in the large
// tiles, unpack them in registers and store them with tcgen05.st; no dequantized operand passes
// through shared memory or HBM. (Through shared memory the 16-bit
// operand would be written and read once per tile, four times the 4-bit codes' bytes each way,
// which bounds a decoding batch before HBM does.) X comes by TMA. Unpacking keeps k in its
// order: bytes of codes are spread to 16-bit halves by a byte permute, where a small integer c
// is the bf16 number c * 2^-133 (subnormals, and the first binade for c >= 128), and one
// bf16 fused multiply-add, c * 2^-133 * 2^127 - zero * 2^-6, leaves (code - zero) * 2^-6
// exactly; 64 goes into the scale. At 4 bits that is 11 instructions per 8 codes.
// Every product with a bf16 token is exact in fp32. The sum of a group (or of up to 128 columns
// of it) leaves tensor memory through the epilogue warps, which add it times the row's scale, a
// value per lane, in fp32.
//
//   warp 0       TMA producer of X, 128 columns a slot
//   warp 1       MMA issuer
//   warp 2       TMA producer of the packed codes (a lane reading its own row from global memory
//                touches a cache line per 16 bytes: 32 per load, which paced the unpacking)
//   warps 4 ...  unpack: sets of four (a warp per 32 tensor-memory lanes), 128-column blocks in turn
//   last eight   epilogue: per unit N / 2 accumulators a thread
//
// Up to 256 tokens (N <= 64): a cluster of CTAs splits d for one tile; each member ends with a share
// of the rows, whose sums the others write into its shared memory, and adds B[a] U there (one dot
// product of `rank` values per output). Many tokens (N = 256): a persistent CTA per SM; the
// adapters are further units of the same product, A = B[a]'s rows, B = U as two bf16 parts
// (high and low, so the sum keeps 16 bits of U), one unit per run of tokens with one adapter,
// which the epilogue adds to that run's columns only.
//
// Bound: HBM bandwidth for few tokens (the codes), the tensor cores for many. Measured at 4 bits, rank
// 16: 4096 x 4096, 1 token 12.3 us, 3001 tokens 123 us (817 TFLOP/s, 42 % of the library GEMM's rate: an
// accumulator leaves tensor memory per 128 columns); 8192 x 8192, 48 tokens 31 us (2.1 TB/s; instruction
// issue 61 % busy, about a fifth of it unpacking).
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "elem.cuh"
#include "packed.cuh"
#include "ring.h"

namespace gptq {

namespace adp {

// ---------------------------------------------------------------------------------
// U = alpha A X
constexpr int SH_WARPS = 8, SH_TOK = 16;
constexpr float kBf16Max = 3.3895314e38f;
// Tokens up to which each reads its adapter by itself: the other kernel reads an adapter once for up to
// 16 tokens that share it, but a group's adapters one after another. m = d = 8192, 128 tokens, the whole
// call, in us: 64 adapters in any order 61 / 227, sorted 66 / 170, 4 adapters sorted 59 / 47.
constexpr int SH_FEW = 256;
// Tokens above which a call may take tiles of 256 tokens, whose adapters' units need U as two bf16
// parts: only the other kernel writes those.
constexpr int TILES_FEW = 256;
static_assert(SH_FEW <= TILES_FEW, "adapter_shrink_few_kernel writes U in fp32 alone");

struct ShrinkParams {
  const uint16_t* X;
  const uint16_t* A;
  const float* alpha;
  const int* ids;
  long long ldx, n_adapters;
  int T, d, rank, splits;
  float* part;                 // [T][rank] fp32, or NULL and
  __nv_bfloat16* hl;           // [T][2 rank], high parts, low parts
};

__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(v)
               : "r"(addr), "r"(rank));
  return v;
}

__device__ __forceinline__ uint32_t map_cluster(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Few tokens: a cluster per token and 16 rows of its adapter, a slice of d per CTA, its warps over
// the rows, four 16-byte loads of a row in flight per lane; the token's piece stays in registers.
// The first CTA adds the slices' sums.
constexpr int SL_COLS = 1024, SH_ROWS = 16;              // columns of a piece, rows of a cluster
__global__ void __launch_bounds__(SH_WARPS * 32) adapter_shrink_few_kernel(ShrinkParams p, int* __restrict__ err) {
  __shared__ float sums[SH_ROWS];
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (p.rank + SH_ROWS - 1) / SH_ROWS, t = blockIdx.y / groups, r0 = (blockIdx.y - t * groups) * SH_ROWS;
  const int nr = min(SH_ROWS, p.rank - r0);                // this cluster's rows
  const int a = p.ids[t];
  if (a >= p.n_adapters && blockIdx.x == 0 && threadIdx.x == 0) report_device_error(err, DEVERR_INDEX);
  const bool has = a >= 0 && a < p.n_adapters;
  const int n8 = p.d / 8, c0 = (int)((long long)n8 * blockIdx.x / p.splits), c1 = (int)((long long)n8 * (blockIdx.x + 1) / p.splits);
  if (has) {
    constexpr int J = SL_COLS / 256;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const uint4* ar = reinterpret_cast<const uint4*>(p.A + (long long)a * p.rank * p.d);
    const float al = p.alpha ? p.alpha[a] : 1.0f;
    for (int s0 = c0; s0 < c1; s0 += SL_COLS / 8) {
      uint4 x[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = s0 + lane + 32 * j;
        x[j] = c < c1 ? reinterpret_cast<const uint4*>(p.X + (long long)t * p.ldx)[c] : z;
      }
#pragma unroll 2
      for (int r = warp; r < nr; r += SH_WARPS) {
        uint4 w[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int c = s0 + lane + 32 * j;
          w[j] = c < c1 ? ar[(long long)(r0 + r) * n8 + c] : z;
        }
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          float u[8], v[8];
          unpack8<BF16>(&x[j], u);
          unpack8<BF16>(&w[j], v);
#pragma unroll
          for (int k = 0; k < 8; ++k) s = fmaf(u[k], v[k], s);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) sums[r] = s0 == c0 ? s * al : fmaf(s, al, sums[r]);
      }
    }
  } else {
    for (int r = threadIdx.x; r < nr; r += SH_WARPS * 32) sums[r] = 0.0f;
  }
  __syncthreads();
  __syncwarp();
  cluster_sync();
  if (blockIdx.x == 0 && threadIdx.x < nr) {
    float s = 0.0f;
    for (int k = 0; k < p.splits; ++k) s += ld_cluster(smem_u32(&sums[threadIdx.x]), (uint32_t)k);
    p.part[(long long)t * p.rank + r0 + threadIdx.x] = s;
  }
  __syncwarp();
  cluster_sync();
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Many tokens: a cluster per 16 tokens, its CTAs' warps over d; for each adapter among the tokens NT groups
// of eight of its rows at a time on mma.sync, so neighbours that share an adapter share the
// reads of its rows. A batch of UN 32-column blocks is loaded before the first is multiplied. The
// CTAs add up each other's sums, each a share of them, in a fixed order.
template <int NT>
__global__ void __launch_bounds__(SH_WARPS * 32) adapter_shrink_kernel(ShrinkParams p, int* __restrict__ err) {
  constexpr int UN = 4;
  __shared__ float red[SH_WARPS][SH_TOK][8 * NT + 1], sums[SH_TOK * 8 * NT];
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int parts = p.splits, t0 = (int)(blockIdx.x / parts) * SH_TOK, part = (int)(blockIdx.x % parts);
  int id = -1;
  if (lane < SH_TOK && t0 + lane < p.T) {
    id = p.ids[t0 + lane];
    if (id >= p.n_adapters) {
      report_device_error(err, DEVERR_INDEX);
      id = -1;
    }
  }
  const int ida = __shfl_sync(0xffffffffu, id, g), idb = __shfl_sync(0xffffffffu, id, g + 8);
  // lane (g, t) holds columns 8 t ... 8 t + 7 of a block: two MMAs' k in a fixed order, the
  // same for both operands. Tokens past the end repeat the last one.
  const int nb = p.d / 32, w0 = SH_WARPS * part + warp, nw = SH_WARPS * parts;
  const int b0 = (int)((long long)nb * w0 / nw), b1 = (int)((long long)nb * (w0 + 1) / nw);     // this warp's blocks
  const uint16_t* xa = p.X + (long long)min(t0 + g, p.T - 1) * p.ldx + 8 * t;
  const uint16_t* xb = p.X + (long long)min(t0 + g + 8, p.T - 1) * p.ldx + 8 * t;
  for (int r0 = 0; r0 < p.rank; r0 += 8 * NT) {
    const int nr = min(8 * NT, p.rank - r0);
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    unsigned todo = __ballot_sync(0xffffffffu, id >= 0);
    while (todo) {
      const int a = __shfl_sync(0xffffffffu, id, __ffs(todo) - 1);
      todo &= ~__ballot_sync(0xffffffffu, id == a);
      const uint16_t* ap[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n)             // rows past the rank repeat the first: their sums are not used
        ap[n] = p.A + ((long long)a * p.rank + r0 + (8 * n < nr ? 8 * n : 0) + g) * p.d + 8 * t;
      float c[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] = 0.0f;
      for (int b = b0; b < b1; b += UN) {
        uint4 u[UN], v[UN], w[UN][NT];
#pragma unroll
        for (int k = 0; k < UN; ++k) {
          const int bk = b + k;
          u[k] = v[k] = make_uint4(0u, 0u, 0u, 0u);
          if (bk < b1) {
            u[k] = *reinterpret_cast<const uint4*>(xa + 32 * bk);
            v[k] = *reinterpret_cast<const uint4*>(xb + 32 * bk);
#pragma unroll
            for (int n = 0; n < NT; ++n) w[k][n] = __ldg(reinterpret_cast<const uint4*>(ap[n] + 32 * bk));
          } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) w[k][n] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
#pragma unroll
        for (int k = 0; k < UN; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_bf16(c[n], u[k].x, v[k].x, u[k].y, v[k].y, w[k][n].x, w[k][n].y);
            mma_bf16(c[n], u[k].z, v[k].z, u[k].w, v[k].w, w[k][n].z, w[k][n].w);
          }
      }
      const float al = p.alpha ? p.alpha[a] : 1.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (ida == a) { acc[n][0] = c[n][0] * al; acc[n][1] = c[n][1] * al; }
        if (idb == a) { acc[n][2] = c[n][2] * al; acc[n][3] = c[n][3] * al; }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      red[warp][g][8 * n + 2 * t] = acc[n][0];
      red[warp][g][8 * n + 2 * t + 1] = acc[n][1];
      red[warp][g + 8][8 * n + 2 * t] = acc[n][2];
      red[warp][g + 8][8 * n + 2 * t + 1] = acc[n][3];
    }
    __syncthreads();
    for (int x = threadIdx.x; x < SH_TOK * nr; x += SH_WARPS * 32) {
      const int i = x / nr, r = x - i * nr;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < SH_WARPS; ++w) s += red[w][i][r];
      sums[x] = s;
    }
    __syncwarp();
    if (parts > 1) cluster_sync();
    for (int x = SH_WARPS * 32 * part + threadIdx.x; x < SH_TOK * nr; x += SH_WARPS * 32 * parts) {
      const int i = x / nr, r = x - i * nr;
      float s = 0.0f;
      if (parts == 1) s = sums[x];
      else
        for (int k = 0; k < parts; ++k) s += ld_cluster(smem_u32(&sums[x]), (uint32_t)k);
      if (t0 + i < p.T && p.part) {
        p.part[(long long)(t0 + i) * p.rank + r0 + r] = s;
      } else if (t0 + i < p.T) {
        // a finite sum has a finite high part; an infinite one is its high part alone (inf - inf is a NaN)
        const float h = fabsf(s) < CUDART_INF_F ? fminf(fmaxf(__bfloat162float(__float2bfloat16_rn(s)), -kBf16Max), kBf16Max) : s;
        p.hl[(long long)(t0 + i) * (2 * p.rank) + r0 + r] = __float2bfloat16_rn(h);
        p.hl[(long long)(t0 + i) * (2 * p.rank) + p.rank + r0 + r] = __float2bfloat16_rn(h == s ? 0.0f : s - h);
      }
    }
    __syncwarp();
    if (parts > 1) cluster_sync();                         // also: nobody leaves while its sums are read
    else __syncthreads();
  }
}

// ---------------------------------------------------------------------------------
// the packed product
constexpr int XK = 64;                                   // columns of one box of X
constexpr int UNPACK0 = 4, NEPI = 8;                     // first unpacking warp, epilogue warps

struct Params {
  const uint32_t* qweight;
  const float* scales;
  const float* zeros;
  const uint16_t* B;
  const int* ids;              // NULL: no adapters
  const float* part;           // few tokens: U [T][rank]
  void* Y;
  long long ldy, n_adapters;
  int m, d, T, gs, G, wpr, unit, rank;
  long long y_bf16;            // 64 bits for the size of all: 8 bytes less and 48 tokens (8192 x 8192) take 32.8 instead of 30.7 us
  uint32_t gs32_mul;           // ceil(2^32 / (gs / 32)), 0 when gs is 32
  int codes_tma;               // the packed rows meet TMA's 16-byte rules: codes come through shared memory
  int mt, nt, S;               // row tiles, token tiles, CTAs that split d
};

// What follows the product in gptq_linear: Y = act(x_scale[t] * sum + bias) * mul + residual. A kernel of its own
// (P below), so that the product alone is what it was.
struct EpiParams : Params {
  const float* x_scale;        // NULL, or the tokens' scales
  const float* bias;           // NULL, or a row's
  const void* mul;             // NULL, or T x m of Y's type
  const void* residual;        // NULL, or T x m of Y's type
  long long ldm, ldr;
  int act;
  int wait_x;                  // X is widen_kernel's, which may still run
};

// Few tokens: tiles of N = 16, 32 or 64 with four accumulators in turn, four sets of unpacking
// warps. Many: tiles of 256 tokens as two parts, an accumulator each, so a block is unpacked once
// for both and one part's epilogue runs beside the other's MMAs; two sets are enough then, and
// the epilogue's 128 sums a thread take registers from the other warps (setmaxnreg: 128 x 32 +
// 256 x 56 + 256 x 168 = 640 x 96, the registers the block has at launch). Four parts of 64
// columns, measured, take 157 instead of 128 us at 3001 tokens: waiting, fencing and issuing
// cost the MMA warp about 450 cycles a part.
template <int BITS, int N>
struct Cfg {
  static constexpr bool MANY = N == 256;
  static constexpr int PARTS = MANY ? 2 : 1, NP = N / PARTS;        // accumulators of a unit, their columns
  static constexpr int ND = MANY ? 2 : 4;                  // accumulators in all
  static constexpr int SETS = MANY ? 2 : 4, EPI0 = UNPACK0 + 4 * SETS, THREADS = (EPI0 + NEPI) * 32;
  static constexpr int REG_ISSUE = 32, REG_UNPACK = 56, REG_EPI = 168;
  static constexpr int SLOTS = !MANY ? 4 : (BITS == 8 ? 2 : 3);     // blocks in the ring: an A buffer, X, packed codes
  // barriers of the slots that are free again and of the codes that have landed: a set of unpacking warps waits on its own
  // (ring.h). The blocks of a tile's adapters are filled up to a multiple of the sets, so that a set's step stays the same for both.
  static constexpr int BARRIERS = barriers_for(SLOTS, SETS);
  static_assert(8 * (2 * SLOTS + 2 * BARRIERS + 2 * ND + 1) + 8 <= 256, "more barriers than have room");
  static constexpr int ROW_BYTES = 16 * BITS;              // packed codes of a row in one block
  static constexpr int C_BYTES = (BM * ROW_BYTES + 1023) / 1024 * 1024;
  static constexpr int X_BOX = N * XK * 2, X_BYTES = 2 * X_BOX;
  static constexpr int TMEM_A = ND * NP;                   // columns: the accumulators, then the A blocks of 64
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int P_BYTES = MANY ? 0 : N * BM * 4;    // the cluster's sums of this member's rows
  static constexpr int SMEM_FIX = SLOTS * (X_BYTES + C_BYTES) + 1024 + 256 + P_BYTES;
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D (tensor memory) += A (tensor memory) B (shared memory), issued by the lane with `leader` set of a
// converged warp: no branch around it, so its operands stay warp-uniform.
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// The runs of one adapter among a tile's 256 tokens, the same in every warp: next() gives a run's
// columns [c0, c1) and its adapter. Lane l holds the ids of columns l, l + 32, ...
struct Runs {
  static constexpr int K = 8;
  uint32_t starts[K];
  int ids[K], c, n;
  __device__ __forceinline__ void init(const Params& p, int t0, int lane) {
    n = min(32 * K, p.T - t0);
    c = 0;
    int prev = -2;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int t = 32 * k + lane;
      int id = -1;
      if (t < n) {
        id = p.ids[t0 + t];
        if (id < 0 || id >= p.n_adapters) id = -1;
      }
      ids[k] = id;
      int before = __shfl_up_sync(0xffffffffu, id, 1);
      if (lane == 0) before = prev;
      starts[k] = __ballot_sync(0xffffffffu, id != before);
      prev = __shfl_sync(0xffffffffu, id, 31);
    }
  }
  __device__ __forceinline__ bool next(int& c0, int& c1, int& id) {
    while (c < n) {
      c0 = c;
      int e = 32 * K, v = -1;                              // the next start after c
#pragma unroll
      for (int k = K - 1; k >= 0; --k) {
        const uint32_t after = 32 * k > c ? starts[k] : (32 * k + 31 > c ? starts[k] & (0xFFFFFFFEu << (c - 32 * k)) : 0u);
        if (after) e = 32 * k + __ffs(after) - 1;
        const int x = __shfl_sync(0xffffffffu, ids[k], c0 & 31);
        if ((c0 >> 5) == k) v = x;
      }
      c1 = min(e, n);
      c = c1;
      id = v;
      if (id >= 0) return true;
    }
    return false;
  }
};

// One CTA fits an SM (896 threads of 72 registers, or 640 of 96). It has to: two on one SM, from
// clusters that each wait for all their members, could wait for each other's tensor memory.
template <int BITS, int N, typename P>
__global__ void __launch_bounds__(Cfg<BITS, N>::THREADS, 1)
adapter_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_u,
                    const __grid_constant__ CUtensorMap map_c, P p,
                    int* __restrict__ err) {
  using C = Cfg<BITS, N>;
  constexpr bool EPI = std::is_same<P, EpiParams>::value;
  constexpr bool MANY = C::MANY;
  constexpr int SLOTS = C::SLOTS, SETS = C::SETS, EPI0 = C::EPI0, THREADS = C::THREADS, NP = C::NP, PARTS = C::PARTS, ND = C::ND;
  constexpr int NC = NP / 2;                               // columns of an epilogue thread in an accumulator
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* codes = smem + SLOTS * C::X_BYTES;
  // full[i]: slot i's A block is in tensor memory (four warps arrive) and its X in shared memory
  // (the producer arrives, TMA completes); empty[n % BARRIERS]: block n's MMAs are done. c_*: the packed codes.
  uint64_t* full = reinterpret_cast<uint64_t*>(codes + SLOTS * C::C_BYTES);
  uint64_t* empty = full + SLOTS;
  uint64_t* c_full = empty + C::BARRIERS;
  uint64_t* c_empty = c_full + C::BARRIERS;
  uint64_t* d_full = c_empty + SLOTS;
  uint64_t* d_empty = d_full + ND;
  uint64_t* drain = d_empty + ND;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* Ps = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(full) + 256);
  float* Us = Ps + C::P_BYTES / 4;                          // few tokens: U, N x rank

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int b = 0; b < SLOTS; ++b) {
      mbar_init(&full[b], 5);
      mbar_init(&c_empty[b], 4);
    }
    for (int b = 0; b < C::BARRIERS; ++b) {
      mbar_init(&empty[b], 1);
      mbar_init(&c_full[b], 1);
    }
    for (int b = 0; b < ND; ++b) {
      mbar_init(&d_full[b], 1);
      mbar_init(&d_empty[b], NEPI);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_c);
    if (MANY) prefetch_tmap(&map_u);
  }
  if (warp == 1) tmem_alloc(tmem_slot, C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_launch();

  const int S = MANY ? 1 : p.S, rank_c = MANY ? 0 : (int)(blockIdx.x % S);
  const int rows = BM / S, rows_lg = 31 - __clz(rows);     // few tokens: the rows that a member of the cluster ends with
  if (S > 1) cluster_arrive();                             // waited for before anything is written to another member
  bool all_here = false;                                   // this warp has
  const int ntiles = p.mt * p.nt, step = MANY ? (int)gridDim.x : ntiles;       // few tokens: one tile per cluster
  const int tile0 = MANY ? (int)blockIdx.x : (int)(blockIdx.x / S);
  const int nblk = (p.d + KB - 1) / KB, blk0 = (int)((long long)nblk * rank_c / S), blk1 = (int)((long long)nblk * (rank_c + 1) / S);
  const int k_lo = blk0 * KB, k_hi = min(p.d, blk1 * KB);
  const int ad_units = (2 * p.rank + KB - 1) / KB;         // A blocks of one adapter
  constexpr uint32_t IDESC = umma_idesc(/*bf16*/ 1, false, false, BM, NP);
  // Block n's slot is free: the MMAs on block n - SLOTS are done, the use of its barrier before u (none, and a new barrier's
  // parity, for the first blocks).
  auto slot_free = [&](uint32_t n) -> bool {
    const uint32_t u = n + (C::BARRIERS - SLOTS);
    return mbar_wait_bounded(&empty[u % C::BARRIERS], ((u / C::BARRIERS) & 1u) ^ 1u, abort_flag);
  };

  if (warp < UNPACK0) {
    if (MANY) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_ISSUE));
    if (warp == 0) {
    // ---------------- TMA producer of X (and of U) ----------------
    uint32_t ab = 0;                                       // blocks so far
    bool ok = true, waited = false;
    if constexpr (EPI) {
      if (p.wait_x) grid_dep_wait();
    }
    // a block of `cols` columns from k on: one box, or two, or none
    auto push = [&](const CUtensorMap* map, int k, int cols, int t) {
      const uint32_t i = ab % SLOTS;
      if (!slot_free(ab)) { ok = false; return; }
      if (cols <= 0) {
        if (lane == 0) mbar_arrive(&full[i]);
      } else if (lane == 0) {
        mbar_arrive_expect_tx(&full[i], cols > XK ? C::X_BYTES : C::X_BOX);
        tma_load_2d(smem + i * C::X_BYTES, map, &full[i], k, t);
        if (cols > XK) tma_load_2d(smem + i * C::X_BYTES + C::X_BOX, map, &full[i], k + XK, t);
      }
      ++ab;
    };
    for (int tile = tile0; ok && tile < ntiles; tile += step) {
      const int t0 = (tile / p.mt) * N;
      for (int k = k_lo; ok && k < k_hi; k += KB) push(&map_x, k, k_hi - k, t0);
      if (MANY && p.ids) {
        if (!waited) { grid_dep_wait(); waited = true; }   // U is the launch before's
        Runs runs;
        runs.init(p, t0, lane);
        int c0, c1, id;
        const uint32_t ab0 = ab;
        while (ok && runs.next(c0, c1, id))
          for (int k = 0; ok && k < 2 * p.rank; k += KB) push(&map_u, k, 2 * p.rank - k, t0);
        while (ok && (ab - ab0) % SETS) push(&map_u, 0, 0, t0);
      }
    }
    if (!ok) { *abort_flag = 1; if (lane == 0) report_device_error(err, DEVERR_TIMEOUT); }
    // copies still in flight when something gave up: their slots' barriers, whose other arrivals may never
    // come then, so with a limit of 1 ms and whatever the abort flag says
    for (uint32_t u = ab > SLOTS ? ab - SLOTS : 0; u < ab; ++u)
      mbar_wait_bounded(&full[u % SLOTS], (u / SLOTS) & 1u, nullptr, 1000000ull);
    } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    uint32_t ab = 0, unit_no = 0;
    bool ok = true;
    const uint32_t leader = elect_leader();
    const uint64_t b_desc0 = umma_sdesc_sw128(smem_u32(smem), 16, 1024);
    // Columns [0, len) of one A operand in blocks of KB and units of `unit`. The warp shares its
    // scheduler with six busy ones, so a block has as few instructions here as it can: two
    // waits, one fence (a fence between the MMAs of one sum makes each wait for the one
    // before: 500 cycles an MMA), eight MMAs, two commits.
    auto stream = [&](int len, int unit) {
      for (int k0 = 0; ok && k0 < len; k0 += KB, ++ab) {
        const int kn = min(KB, len - k0);
        const uint32_t i = ab % SLOTS, at = tmem + C::TMEM_A + i * (KB / 2);
        const uint64_t bd = b_desc0 + (uint64_t)(i * (C::X_BYTES / 16));
        if (!mbar_wait_poll(&full[i], (ab / SLOTS) & 1u, abort_flag)) { ok = false; break; }
        if (unit == KB && kn == KB) {
#pragma unroll
          for (int h = 0; h < PARTS; ++h, ++unit_no) {
            const uint32_t buf = unit_no % ND, dt = tmem + buf * NP;
            if (!mbar_wait_poll(&d_empty[buf], ((unit_no / ND) & 1u) ^ 1u, abort_flag)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_f16_ta(dt, at + 8 * kk, bd + (h * NP * XK * 2 + (kk >= 4 ? C::X_BOX : 0)) / 16 + 2 * (kk & 3), IDESC, kk != 0,
                          leader);
            umma_commit_by(&d_full[buf], leader);
          }
        } else {
          for (int u = 0; ok && u < kn; u += unit) {
            for (int h = 0; h < PARTS; ++h, ++unit_no) {
              const uint32_t buf = unit_no % ND;
              if (!mbar_wait_poll(&d_empty[buf], ((unit_no / ND) & 1u) ^ 1u, abort_flag)) { ok = false; break; }
              tc_fence_after();
              for (int k = u; k < min(u + unit, kn); k += 16)
                umma_f16_ta(tmem + buf * NP, at + k / 2, bd + (h * NP * XK * 2 + (k >= XK ? C::X_BOX : 0)) / 16 + (k & (XK - 1)) / 8,
                            IDESC, k != u, leader);
              umma_commit_by(&d_full[buf], leader);
            }
          }
        }
        if (!ok) break;
        umma_commit_by(&empty[ab % C::BARRIERS], leader);
      }
    };
    for (int tile = tile0; ok && tile < ntiles; tile += step) {
      stream(k_hi - k_lo, p.unit);
      if (MANY && p.ids) {
        Runs runs;
        runs.init(p, (tile / p.mt) * N, lane);
        int c0, c1, id;
        const uint32_t ab0 = ab;
        while (ok && runs.next(c0, c1, id)) stream(2 * p.rank, KB);
        for (; ok && (ab - ab0) % SETS; ++ab) {
          if (!mbar_wait_poll(&full[ab % SLOTS], (ab / SLOTS) & 1u, abort_flag)) { ok = false; break; }
          umma_commit_by(&empty[ab % C::BARRIERS], leader);
        }
      }
    }
    if (!ok) { *abort_flag = 1; if (lane == 0) report_device_error(err, DEVERR_TIMEOUT); }
    umma_commit_by(drain, leader);
    mbar_wait_bounded(drain, 0, nullptr);
    } else if (warp == 2 && p.codes_tma) {
    // ---------------- TMA producer of the packed codes ----------------
    uint32_t cn = 0;
    bool ok = true;
    for (int tile = tile0; ok && tile < ntiles; tile += step) {
      const int r0 = (tile % p.mt) * BM;
      for (int b = blk0; b < blk1; ++b, ++cn) {
        const uint32_t i = cn % SLOTS;
        if (!mbar_wait_bounded(&c_empty[i], ((cn / SLOTS) & 1u) ^ 1u, abort_flag)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(&c_full[cn % C::BARRIERS], BM * C::ROW_BYTES);
          tma_load_2d(codes + i * C::C_BYTES, &map_c, &c_full[cn % C::BARRIERS], b * C::ROW_BYTES, r0);
        }
      }
    }
    if (!ok) { *abort_flag = 1; if (lane == 0) report_device_error(err, DEVERR_TIMEOUT); }
    for (uint32_t u = cn > SLOTS ? cn - SLOTS : 0; u < cn; ++u) mbar_wait_bounded(&c_full[u % C::BARRIERS], (u / C::BARRIERS) & 1u, nullptr);
    } else if (warp == 3 && !MANY && p.ids) {
    // ---------------- U, while the others work ----------------
    grid_dep_wait();
    const int t0 = (tile0 / p.mt) * N, n4 = min(N, p.T - t0) * p.rank / 4;
    const float4* u = reinterpret_cast<const float4*>(p.part + (long long)t0 * p.rank);
#pragma unroll 4
    for (int x = lane; x < n4; x += 32) reinterpret_cast<float4*>(Us)[x] = u[x];
    }
  } else if (warp < EPI0) {
    // ---------------- unpack: words -> registers -> tensor memory ----------------
    if (MANY) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_UNPACK));
    constexpr int W32 = BITS, WB = 4 * W32;                // words of 32 columns, of a block
    const int set = (warp - UNPACK0) >> 2, q = warp & 3, row_l = 32 * q + lane;
    const uint32_t ta0 = tmem + ((uint32_t)(32 * q) << 16) + C::TMEM_A;
    const bool one_zero = p.gs % KB == 0;
    auto group_of = [&](int c32) -> int {                  // the group of columns 32 c32 ...
      return p.gs32_mul ? (int)__umulhi((uint32_t)c32, p.gs32_mul) : c32;
    };
    uint32_t ab = 0, cb0 = 0;                              // A blocks and stages of codes so far, all sets'
    bool ok = true;
    uint32_t ta = 0;
    auto ready = [&]() -> bool {                           // the block's buffer is free
      ta = ta0 + (ab % SLOTS) * (KB / 2);
      if (!slot_free(ab)) {
        *abort_flag = 1;
        if (lane == 0) report_device_error(err, DEVERR_TIMEOUT);
        return false;
      }
      tc_fence_after();
      return true;
    };
    auto publish = [&]() {
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[ab % SLOTS]);
    };
    for (int tile = tile0; ok && tile < ntiles; tile += step) {
      const int row = (tile % p.mt) * BM + row_l;
      const bool live = row < p.m;
      const float* zr = p.zeros + (long long)(live ? row : 0) * p.G;
      // this set's blocks: first, first + SETS, ... (ab counts every set's, to the tile's end)
      const uint32_t ab0 = ab;
      const int first = blk0 + (int)((set - ab0) % SETS);
      const uint32_t* wp = p.qweight + (long long)(live ? row : 0) * p.wpr + (long long)first * WB;
      float z = 0.0f;
      if (one_zero && first < blk1) z = __ldg(zr + group_of(4 * first));
      for (int b = first; b < blk1; b += SETS) {
        ab = ab0 + (uint32_t)(b - blk0);
        uint32_t w[WB];
        if (p.codes_tma) {
          const uint32_t cn = cb0 + (uint32_t)(b - blk0), st = cn % SLOTS;
          if (!mbar_wait_bounded(&c_full[cn % C::BARRIERS], (cn / C::BARRIERS) & 1u, abort_flag)) {
            *abort_flag = 1;
            if (lane == 0) report_device_error(err, DEVERR_TIMEOUT);
            ok = false;
            break;
          }
          const uint32_t sc = smem_u32(codes) + st * C::C_BYTES;
#pragma unroll
          for (int i = 0; i < BITS; ++i) lds_piece<BITS>(sc, row_l, i, w + 4 * i);
          // without the fence the next copy could overwrite words that a lane's load had not read yet
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c_empty[st]);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (b * KB + 32 * c < p.d) load_words<W32>(wp + c * W32, w + c * W32);
          wp += SETS * WB;
        }
        const uint32_t nzb = neg_zero(z);
        if (one_zero && b + SETS < blk1) z = __ldg(zr + group_of(4 * (b + SETS)));
        if (!ready()) { ok = false; break; }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (b * KB + 32 * c < p.d) {
            const uint32_t nz = one_zero ? nzb : neg_zero(__ldg(zr + group_of(4 * b + c)));
            uint32_t o[16];
            unpack32<BITS>(w + c * W32, nz, o);
            tmem_st16(ta + 16 * c, o);
          }
        }
        publish();
      }
      cb0 += (uint32_t)(blk1 - blk0);
      ab = ab0 + (uint32_t)(blk1 - blk0);
      if (MANY && p.ids) {
        // the adapters' rows as further A blocks: column k is B[a][row][k mod rank]
        Runs runs;
        runs.init(p, (tile / p.mt) * N, lane);
        int c0, c1, id;
        const uint32_t first_ad = ab;
        while (ok && runs.next(c0, c1, id)) {
          const uint32_t* br = reinterpret_cast<const uint32_t*>(p.B + ((long long)id * p.m + (live ? row : 0)) * p.rank);
          for (int u = 0; u < ad_units; ++u, ++ab) {
            if ((int)(ab % SETS) != set) continue;
            if (!ready()) { ok = false; break; }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (u * KB + 32 * c < 2 * p.rank) {
                uint32_t o[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4) {          // eight columns, one 16-byte load (rank % 8 == 0)
                  const int k = u * KB + 32 * c + 2 * i;
                  const uint4 v = k < 2 * p.rank ? __ldg(reinterpret_cast<const uint4*>(br + (k >= p.rank ? k - p.rank : k) / 2))
                                                 : make_uint4(0u, 0u, 0u, 0u);
                  o[i] = v.x; o[i + 1] = v.y; o[i + 2] = v.z; o[i + 3] = v.w;
                }
                tmem_st16(ta + 16 * c, o);
              }
            }
            publish();
          }
        }
        for (; ok && (ab - first_ad) % SETS; ++ab) {
          if ((int)(ab % SETS) != set) continue;
          if (!ready()) { ok = false; break; }
          if (lane == 0) mbar_arrive(&full[ab % SLOTS]);
        }
      }
    }
  } else {
    // ---------------- epilogue ----------------
    if (MANY) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REG_EPI));
    const int q = warp & 3, h = (warp - EPI0) >> 2;
    const uint32_t td = tmem + ((uint32_t)(32 * q) << 16) + h * NC;
    uint32_t unit_no = 0;
    bool ok = true;
    constexpr int LD = NC < 16 ? 8 : 16;
    for (int tile = tile0; ok && tile < ntiles; tile += step) {
      const int row = (tile % p.mt) * BM + 32 * q + lane, t0 = (tile / p.mt) * N;
      const float* sr = p.scales + (long long)(row < p.m ? row : 0) * p.G;
      uint64_t run[PARTS][NC / 2];                        // fp32 pairs
#pragma unroll
      for (int x = 0; x < PARTS; ++x)
#pragma unroll
        for (int c = 0; c < NC / 2; ++c) run[x][c] = 0ull;
      auto wait = [&]() -> bool {
        if (!mbar_wait_bounded(&d_full[unit_no % ND], (unit_no / ND) & 1u, abort_flag)) {
          *abort_flag = 1;
          if (lane == 0) report_device_error(err, DEVERR_TIMEOUT);
          return false;
        }
        tc_fence_after();
        return true;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_empty[unit_no % ND]);
        ++unit_no;
      };
      int grp = k_lo / p.gs, kg = k_lo - grp * p.gs;
      // a lane's row of scales is its own cache line: four at a time where they are aligned
      const bool by4 = (p.G & 3) == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 15) == 0;
      float4 s4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float sn = 0.0f;
      auto next_scale = [&](bool begin) {
        if (by4) {
          if (begin || (grp & 3) == 0) s4 = __ldg(reinterpret_cast<const float4*>(sr + (grp & ~3)));
        } else {
          sn = __ldg(sr + grp);
        }
      };
      if (k_lo < k_hi) next_scale(true);
      for (int k = k_lo; k < k_hi; k += p.unit) {
        const float s = 64.0f * (by4 ? ((grp & 2) ? ((grp & 1) ? s4.w : s4.z) : ((grp & 1) ? s4.y : s4.x)) : sn);
        kg += p.unit;
        if (kg >= p.gs) {
          kg = 0;
          ++grp;
          if (k + p.unit < k_hi) next_scale(false);
        }
        const uint64_t ss = pack2(s, s);
#pragma unroll
        for (int x = 0; x < PARTS; ++x) {
          if (!wait()) { ok = false; break; }
#pragma unroll
          for (int c = 0; c < NC; c += LD) {
            uint32_t a[LD];
            tmem_ld<LD>(td + (unit_no % ND) * NP + c, a);
            tmem_ld_wait<LD>(a);
#pragma unroll
            for (int i = 0; i < LD; i += 2) run[x][(c + i) / 2] = fma2(pack2u(a[i], a[i + 1]), ss, run[x][(c + i) / 2]);
          }
          release();
        }
        if (!ok) break;
      }
      if (MANY) {
        if (p.ids) {
          Runs runs;
          runs.init(p, t0, lane);
          int c0, c1, id;
          while (ok && runs.next(c0, c1, id)) {
            for (int u = 0; ok && u < ad_units; ++u) {
#pragma unroll
              for (int x = 0; x < PARTS; ++x) {
                if (!wait()) { ok = false; break; }
                const int base = x * NP + h * NC;          // the run's columns among this thread's
                if (c0 < base + NC && c1 > base) {
#pragma unroll
                  for (int c = 0; c < NC; c += LD) {
                    uint32_t a[LD];
                    tmem_ld<LD>(td + (unit_no % ND) * NP + c, a);
                    tmem_ld_wait<LD>(a);
#pragma unroll
                    for (int i = 0; i < LD; i += 2) {
                      const bool in0 = base + c + i >= c0 && base + c + i < c1, in1 = base + c + i + 1 >= c0 && base + c + i + 1 < c1;
                      run[x][(c + i) / 2] = add2(pack2u(in0 ? a[i] : 0u, in1 ? a[i + 1] : 0u), run[x][(c + i) / 2]);
                    }
                  }
                }
                release();
              }
            }
          }
        }
        if (ok && row < p.m) {
#pragma unroll
          for (int x = 0; x < PARTS; ++x)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const int t = t0 + x * NP + h * NC + c;
              const float v = half2f(run[x][c / 2], c & 1);
              if (t < p.T) {
                if (p.y_bf16) reinterpret_cast<__nv_bfloat16*>(p.Y)[(long long)t * p.ldy + row] = __float2bfloat16_rn(v);
                else reinterpret_cast<float*>(p.Y)[(long long)t * p.ldy + row] = v;
              }
            }
        }
      } else {
        // each row's sums to the member that ends with it: [member][token][row]
        const int own = (32 * q + lane) >> rows_lg;
        uint32_t to = smem_u32(Ps) + 4 * (((rank_c * N) << rows_lg) + ((32 * q + lane) & (rows - 1)));
        if (S > 1) {
          __syncwarp();
          cluster_wait();
          all_here = true;
          to = map_cluster(to, (uint32_t)own);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float v = half2f(run[0][c / 2], c & 1);
          const uint32_t at = to + 4 * ((h * NC + c) << rows_lg);
          if (S > 1) st_cluster(at, v); else asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
        }
      }
    }
  }

  if (!MANY) {
    // ---- few tokens: the cluster's sums, each member its share of the rows. The adapters' dot
    // products come first: they wait for no other CTA.
    const int t0 = (tile0 / p.mt) * N, r0 = (tile0 % p.mt) * BM;
    const int nout = rows * min(N, p.T - t0);
    if (S > 1) {                                           // the members' sums are written
      __syncwarp();
      if (!all_here) cluster_wait();
      cluster_arrive();
    }
    // 2^lg lanes share an output: each takes every 2^lg-th 16 bytes of the adapter's row and member
    // of the cluster, so an output's loads are in flight together
    // (as many as leave one pass over the outputs: 48 tokens, 8192 x 8192, rank 16: 28.5 us with two, 27.2 with one)
    constexpr int OUT = 4;                                 // outputs of a thread in flight
    int lg = p.ids ? min(3, 31 - __clz(p.rank / 8)) : 0;
    while (lg > 0 && nout << lg > OUT * THREADS) --lg;
    const int part = lane & ((1 << lg) - 1);
    bool met = false;
    for (int x0 = threadIdx.x; x0 - lane < nout << lg || !met; x0 += OUT * THREADS) {
      float sum[OUT];
      int col[OUT], rl[OUT];                               // token of the tile (-1: none), row of the tile
      const uint16_t* br[OUT];                             // the adapter's row
#pragma unroll
      for (int o = 0; o < OUT; ++o) {
        const int x = (x0 + o * THREADS) >> lg;
        col[o] = x < nout ? x >> rows_lg : -1;
        rl[o] = (rank_c << rows_lg) + (x & (rows - 1));
        if (r0 + rl[o] >= p.m) col[o] = -1;
        sum[o] = 0.0f;
        br[o] = nullptr;
        if (p.ids && col[o] >= 0) {
          const int id = p.ids[t0 + col[o]];
          if (id >= 0 && id < p.n_adapters) br[o] = p.B + ((long long)id * p.m + r0 + rl[o]) * p.rank;
        }
      }
      auto load = [&](uint4 (&v)[OUT], int r) {
#pragma unroll
        for (int o = 0; o < OUT; ++o) {
          v[o] = make_uint4(0u, 0u, 0u, 0u);
          if (br[o] && r < p.rank) v[o] = __ldg(reinterpret_cast<const uint4*>(br[o] + r));
        }
      };
      uint4 bv[OUT];
      load(bv, 8 * part);
      // the first rows are on their way while the others finish; then U is in shared memory (warp 3)
      if (!met) __syncthreads();
      if (p.ids) {
        for (int r = 8 * part; r < p.rank; r += 8 << lg) {
          uint4 next[OUT];
          load(next, r + (8 << lg));
#pragma unroll
          for (int o = 0; o < OUT; ++o) {
            if (br[o]) {
              float v[8];
              unpack8<BF16>(&bv[o], v);
              const float* u = Us + col[o] * p.rank + r;
              const float4 ua = *reinterpret_cast<const float4*>(u), ub = *reinterpret_cast<const float4*>(u + 4);
              sum[o] = fmaf(v[0], ua.x, sum[o]); sum[o] = fmaf(v[1], ua.y, sum[o]);
              sum[o] = fmaf(v[2], ua.z, sum[o]); sum[o] = fmaf(v[3], ua.w, sum[o]);
              sum[o] = fmaf(v[4], ub.x, sum[o]); sum[o] = fmaf(v[5], ub.y, sum[o]);
              sum[o] = fmaf(v[6], ub.z, sum[o]); sum[o] = fmaf(v[7], ub.w, sum[o]);
            }
            bv[o] = next[o];
          }
        }
      }
      __syncwarp();
      if (!met && S > 1) cluster_wait();
      met = true;
      for (int k = part; k < S; k += 1 << lg) {
        float v[OUT];
#pragma unroll
        for (int o = 0; o < OUT; ++o) {
          v[o] = 0.0f;
          if (col[o] < 0) continue;
          v[o] = Ps[((k * N + col[o]) << rows_lg) + (rl[o] & (rows - 1))];
        }
#pragma unroll
        for (int o = 0; o < OUT; ++o) sum[o] += v[o];
      }
      __syncwarp();
#pragma unroll
      for (int o = 0; o < OUT; ++o) {
        for (int k = 0; k < lg; ++k) sum[o] += __shfl_xor_sync(0xffffffffu, sum[o], 1 << k);
        if (col[o] < 0 || part) continue;
        const long long at = (long long)(t0 + col[o]) * p.ldy + r0 + rl[o];
        if constexpr (EPI) {
          const long long t = t0 + col[o], r = r0 + rl[o];
          const float mul = p.mul ? read_y(p.mul, t * p.ldm + r, p.y_bf16) : 1.0f;
          const float res = p.residual ? read_y(p.residual, t * p.ldr + r, p.y_bf16) : 0.0f;
          float v = activate(fmaf(sum[o], p.x_scale ? p.x_scale[t] : 1.0f, p.bias ? p.bias[r] : 0.0f), p.act);
          if (p.mul) v *= mul;
          if (p.residual) v += res;
          sum[o] = v;
        }
        if (p.y_bf16) reinterpret_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(sum[o]);
        else reinterpret_cast<float*>(p.Y)[at] = sum[o];
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

bool make_map(CUtensorMap* m, const void* base, long long inner, long long outer, long long ld, int rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {XK, (cuuint32_t)rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// How a call of T tokens is cut. Up to 256 tokens: tiles of up to 64, with clusters that split d so
// that about every SM has a CTA. More: tiles of 256 once there are more tiles of 64 than SMs.
// Measured at 4 bits, in us, 64 / 256: m = d = 8192, 512 tokens 172 / 80; m = d = 4096, 768 tokens 90 / 49.
// In tiles of 256 every run of tokens with one adapter is a unit of the product: for prompts a few, for
// a decoding batch up to one per token. So up to 256 tokens, which may be such a batch, stay with tiles
// of 64: of 64 adapters in any order, m = d = 8192, 256 tokens take 104 / 575 (sorted, of 4: 102 / 78). (512
// tokens of 64 adapters in any order take 597, sorted 160: the caller of long batches sorts them.)
struct Plan {
  int N, mt, nt, S, splits;
};
Plan plan_of(long long m, long long d, long long T, int rank) {
  Plan p;
  const int sms = sm_count();
  p.mt = (int)((m + BM - 1) / BM);
  p.S = 1;
  p.splits = 1;
  if (T > TILES_FEW && p.mt * ((T + 63) / 64) > sms) {
    p.N = 256;
  } else {
    p.N = T <= 16 ? 16 : (T <= 32 ? 32 : 64);
    const long long few = (long long)p.mt * ((T + p.N - 1) / p.N);
    while (p.S < 8 && 2 * p.S * few <= sms && 2 * p.S * KB <= d) p.S *= 2;
  }
  p.nt = (int)((T + p.N - 1) / p.N);
  // slices of d for U, a cluster's CTAs, of at least 256 columns each
  if (T <= SH_FEW) {
    const long long clusters = T * ((rank + SH_ROWS - 1) / SH_ROWS);
    while (p.splits < 8 && p.splits * 512 <= d && clusters * p.splits < 2 * sms) p.splits *= 2;
  } else {
    // U's CTAs on SMs that the product leaves free run beside it; on the others they hold it up. So
    // as many slices as fit there when they are done before the product (a slice of U takes about
    // as long as a tile of 64 tokens over as many columns), else as many as make U itself quick.
    // Measured at 4 bits, d = 8192, rank 16, in us, free SMs only / all: m = 8192, 384 tokens 74 / 82;
    // m = 1024, 768 tokens 47 / 53. Too few are free: m = 1024, 1024 tokens 72 / 55; m = 8192, 1024 tokens
    // 156 / 139.
    const long long groups = (T + SH_TOK - 1) / SH_TOK, room = sms - (long long)p.mt * p.nt * p.S;
    while (p.splits < 8 && p.splits * 512 <= d && 2 * p.splits * groups <= room) p.splits *= 2;
    if (groups > room || p.splits < p.S)
      while (p.splits < 8 && p.splits * 512 <= d && 2 * p.splits * groups <= 4 * sms) p.splits *= 2;
  }
  return p;
}

template <int BITS, int N, typename P>
gptq_status launch(const CUtensorMap& mx, const CUtensorMap& mu, P p, bool pdl, cudaStream_t s) {
  CUtensorMap mc = mx;
  p.codes_tma = make_code_map(&mc, p.qweight, p.m, (long long)p.wpr * 4, BITS) ? 1 : 0;
  using C = Cfg<BITS, N>;
  const size_t smem = C::SMEM_FIX + (C::MANY ? 0 : (size_t)N * p.rank * 4);
  static PerDevice done;
  const size_t most = C::SMEM_FIX + (C::MANY ? 0 : (size_t)N * 128 * 4);
  if (gptq_status st = allow_smem(done, adapter_gemm_kernel<BITS, N, P>, most, "adapter_gemm_kernel")) return st;
  const long long tiles = (long long)p.mt * p.nt;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(C::MANY ? std::min<long long>(tiles, sm_count()) : tiles * p.S));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int na = 0;
  attr[na].id = cudaLaunchAttributeClusterDimension;
  attr[na].val.clusterDim.x = (unsigned)(C::MANY ? 1 : p.S);
  attr[na].val.clusterDim.y = 1;
  attr[na].val.clusterDim.z = 1;
  ++na;
  if (pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  cudaLaunchKernelEx(&cfg, adapter_gemm_kernel<BITS, N, P>, mx, mu, mc, p, device_error_word());
  count_launch();
  return check_launch("adapter_gemm_kernel");
}

template <int BITS, typename P>
gptq_status launch_n(int N, const CUtensorMap& mx, const CUtensorMap& mu, const P& p, bool pdl, cudaStream_t s) {
  switch (N) {
    case 16: return launch<BITS, 16, P>(mx, mu, p, pdl, s);
    case 32: return launch<BITS, 32, P>(mx, mu, p, pdl, s);
    case 64: return launch<BITS, 64, P>(mx, mu, p, pdl, s);
    default:
      if constexpr (std::is_same<P, Params>::value) return launch<BITS, 256, P>(mx, mu, p, pdl, s);
      else return set_error(GPTQ_ERR_UNSUPPORTED, "what follows the product of many tokens is a kernel of its own");
  }
}

}  // namespace adp

// Workspace: U, in fp32 or as two bf16 parts.
size_t adapter_workspace_bytes(long long m, long long d, int bits, int group_size, long long T, int rank) {
  using namespace adp;
  (void)bits;
  (void)group_size;
  (void)m;
  (void)d;
  return round256(4 * (size_t)std::max(1LL, T) * rank);
}

namespace adp {
// p: what follows the product, or an empty Params
template <typename P>
gptq_status product_launch(P p, const uint32_t* qweight, const float* scales, const float* zeros, long long m, long long d, int bits,
                           int group_size, const uint16_t* X, long long T, long long ldx, const uint16_t* A, const uint16_t* B,
                           const float* alpha, long long n_adapters, int rank, const int* ids, void* Y, int y_dtype, long long ldy,
                           void* ws, cudaStream_t s) {
  const Plan pl = plan_of(m, d, T, rank);
  if ((long long)pl.mt * pl.nt * pl.S > 0x7FFFFFFF) return set_error(GPTQ_ERR_INVALID_ARG, "too many output tiles");
  if (ids) {
    ShrinkParams q{};
    q.X = X; q.A = A; q.alpha = alpha; q.ids = ids; q.ldx = ldx; q.n_adapters = n_adapters;
    q.T = (int)T; q.d = (int)d; q.rank = rank; q.splits = pl.splits;
    if (pl.N == 256) q.hl = reinterpret_cast<__nv_bfloat16*>(ws);
    else q.part = reinterpret_cast<float*>(ws);
    cudaLaunchConfig_t cfg = {};
    // clusters along x where there may be more of them than gridDim.y holds
    const long long few = T * ((rank + SH_ROWS - 1) / SH_ROWS), many = (T + SH_TOK - 1) / SH_TOK;
    cfg.gridDim = T <= SH_FEW ? dim3((unsigned)pl.splits, (unsigned)few) : dim3((unsigned)(pl.splits * many));
    cfg.blockDim = dim3(SH_WARPS * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)pl.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (T <= SH_FEW) cudaLaunchKernelEx(&cfg, adapter_shrink_few_kernel, q, device_error_word());
    else if (rank == 8) cudaLaunchKernelEx(&cfg, adapter_shrink_kernel<1>, q, device_error_word());
    else if (rank == 16) cudaLaunchKernelEx(&cfg, adapter_shrink_kernel<2>, q, device_error_word());
    else cudaLaunchKernelEx(&cfg, adapter_shrink_kernel<4>, q, device_error_word());
    count_launch();
    if (gptq_status st = check_launch("adapter_shrink_kernel")) return st;
  }
  p.qweight = qweight; p.scales = scales; p.zeros = zeros; p.B = B; p.ids = ids; p.part = reinterpret_cast<const float*>(ws);
  p.Y = Y; p.ldy = ldy; p.n_adapters = n_adapters;
  p.m = (int)m; p.d = (int)d; p.T = (int)T;
  p.gs = group_size < 0 ? (int)d : group_size;
  p.G = (int)(d / p.gs);
  p.wpr = (int)(d / 32 * bits);
  const unsigned gs32 = (unsigned)p.gs / 32;
  p.gs32_mul = gs32 == 1 ? 0u : (uint32_t)((0x100000000ULL + gs32 - 1) / gs32);
  p.unit = p.gs % 128 == 0 ? 128 : (p.gs % 64 == 0 ? 64 : 32);
  p.rank = rank; p.y_bf16 = y_dtype == GPTQ_BF16;
  p.mt = pl.mt; p.nt = pl.nt; p.S = pl.S;
  CUtensorMap mx, mu;
  if (!make_map(&mx, X, d, T, ldx, pl.N)) return set_error(GPTQ_ERR_CUDA, "cuTensorMapEncodeTiled failed for X");
  mu = mx;
  if (ids && pl.N == 256 && !make_map(&mu, ws, 2 * rank, T, 2 * rank, pl.N))
    return set_error(GPTQ_ERR_CUDA, "cuTensorMapEncodeTiled failed for the adapters' inner product");
  bool pdl = ids != nullptr;
  if constexpr (std::is_same<P, EpiParams>::value) pdl |= p.wait_x != 0;
  switch (bits) {
    case 2: return launch_n<2>(pl.N, mx, mu, p, pdl, s);
    case 3: return launch_n<3>(pl.N, mx, mu, p, pdl, s);
    case 4: return launch_n<4>(pl.N, mx, mu, p, pdl, s);
    default: return launch_n<8>(pl.N, mx, mu, p, pdl, s);
  }
}

// What follows the product of many tokens with adapters: from its fp32 sums Z (T x m), a row of 256 outputs a block. (In the
// product's own epilogue it took the registers that hold the sums: 11008 x 4096, 3001 tokens, gate 861 us without adapters.)
__global__ void __launch_bounds__(256) follow_kernel(const float* __restrict__ Z, EpiParams p) {
  const long long t = blockIdx.y + (long long)blockIdx.z * gridDim.y;
  const int row = blockIdx.x * 256 + threadIdx.x;
  if (row >= p.m || t >= p.T) return;
  const float mul = p.mul ? read_y(p.mul, t * p.ldm + row, p.y_bf16) : 1.0f;
  const float res = p.residual ? read_y(p.residual, t * p.ldr + row, p.y_bf16) : 0.0f;
  float v = activate(fmaf(Z[t * p.m + row], p.x_scale ? p.x_scale[t] : 1.0f, p.bias ? p.bias[row] : 0.0f), p.act);
  if (p.mul) v *= mul;
  if (p.residual) v += res;
  if (p.y_bf16) reinterpret_cast<__nv_bfloat16*>(p.Y)[t * p.ldy + row] = __float2bfloat16_rn(v);
  else reinterpret_cast<float*>(p.Y)[t * p.ldy + row] = v;
}

// Tokens in e4m3 to bf16, which holds every one of their values; 16 a thread.
__global__ void __launch_bounds__(256) widen_kernel(const uint8_t* __restrict__ x, long long ldx, uint16_t* __restrict__ y, int d, long long n16) {
  grid_dep_launch();
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n16) return;
  const int per = d / 16;
  const long long t = i / per;
  const int c = (int)(i - t * per) * 16;
  const uint4 v = *reinterpret_cast<const uint4*>(x + t * ldx + c);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[k / 2] >> (16 * (k & 1)))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    o[k] = *reinterpret_cast<const uint32_t*>(&b);
  }
  uint4* to = reinterpret_cast<uint4*>(y + t * d + c);
  to[0] = make_uint4(o[0], o[1], o[2], o[3]);
  to[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

}  // namespace adp

gptq_status adapter_linear_launch(const uint32_t* qweight, const float* scales, const float* zeros, long long m,
                                  long long d, int bits, int group_size, const uint16_t* X, long long T, long long ldx,
                                  const uint16_t* A, const uint16_t* B, const float* alpha, long long n_adapters,
                                  int rank, const int* ids, void* Y, int y_dtype, long long ldy, void* ws,
                                  cudaStream_t s) {
  return adp::product_launch(adp::Params{}, qweight, scales, zeros, m, d, bits, group_size, X, T, ldx, A, B, alpha, n_adapters, rank,
                             ids, Y, y_dtype, ldy, ws, s);
}

gptq_status linear_tiles_launch(const uint32_t* qweight, const float* scales, const float* zeros, long long m, long long d,
                                int bits, int group_size, const void* X, bool bytes, long long T, long long ldx,
                                const float* x_scale, const float* bias, int act, const void* mul, long long ldm,
                                const void* residual, long long ldr, void* Y, int y_dtype, long long ldy,
                                cudaStream_t s);           // linear_tiles.cu
gptq_status linear_few_launch(const uint32_t* qweight, const float* scales, const float* zeros, long long m, long long d,
                              int bits, int group_size, const void* X, bool bytes, long long T, long long ldx,
                              const float* x_scale, const float* bias, int act, const void* mul, long long ldm,
                              const void* residual, long long ldr, void* Y, int y_dtype, long long ldy,
                              cudaStream_t s);             // linear_few.cu

constexpr long long FEW = 8;                               // tokens up to which linear_few.cu may take a call
static bool by_few(long long d, int group_size, long long T) {
  return T <= FEW && d % adp::KB == 0 && (group_size < 0 || group_size % adp::KB == 0);
}

// Without adapters, more than 64 tokens may go by linear_tiles.cu, in 8 bits as they are where (code - zero) fits e4m3. A
// block of 128 columns takes either kernel about 0.75 us a tile (of 256 tokens there, of 64 here, in up to eight slices of
// d), so the one with fewer blocks one after another. 11008 x 4096, in us, here / there: 64 tokens 23 / 25, 128 tokens
// 44 / 30, 256 tokens 64 / 31.
static bool by_tiles(long long m, long long d, long long T) {
  if (T <= 64) return false;
  const adp::Plan pl = adp::plan_of(m, d, T, 8);
  if (pl.N == 256) return true;
  const long long sms = sm_count(), blocks = (d + adp::KB - 1) / adp::KB, mt = (m + adp::BM - 1) / adp::BM;
  const long long here = ((long long)pl.mt * pl.nt * pl.S + sms - 1) / sms * ((blocks + pl.S - 1) / pl.S);
  return (mt * ((T + 255) / 256) + sms - 1) / sms * blocks < here;
}

// Workspace: the adapters' U (rank 0: there are none) and many tokens' sums before what follows them, or 8-bit tokens as bf16
// (adapters are refused beside them).
size_t linear_workspace_bytes(long long m, long long d, int bits, int group_size, long long T, int x_dtype, int rank) {
  if (x_dtype != GPTQ_E4M3) {
    if (rank == 0 || T == 0) return 256;
    return adapter_workspace_bytes(m, d, bits, group_size, T, rank) +
           (adp::plan_of(m, d, T, rank).N == 256 ? adp::round256((size_t)T * m * 4) : 0);
  }
  return by_few(d, group_size, T) || (by_tiles(m, d, T) && bits <= 4) ? 256 : adp::round256((size_t)std::max(1LL, T) * d * 2);
}

gptq_status linear_launch(const uint32_t* qweight, const float* scales, const float* zeros, long long m, long long d,
                          int bits, int group_size, const void* X, int x_dtype, long long T, long long ldx,
                          const float* x_scale, const uint16_t* A, const uint16_t* B, const float* alpha,
                          long long n_adapters, int rank, const int* ids, const float* bias, int act, const void* mul,
                          long long ldm, const void* residual, long long ldr, void* Y, int y_dtype, long long ldy,
                          void* ws, cudaStream_t s) {
  using namespace adp;
  if (!ids && by_few(d, group_size, T))
    return linear_few_launch(qweight, scales, zeros, m, d, bits, group_size, X, x_dtype == GPTQ_E4M3, T, ldx, x_scale, bias, act, mul,
                             ldm, residual, ldr, Y, y_dtype, ldy, s);
  const bool tiles = !ids && by_tiles(m, d, T);
  if (!ids) rank = 8;                                      // of no adapter
  const uint16_t* x = reinterpret_cast<const uint16_t*>(X);
  if (x_dtype == GPTQ_E4M3 && !(tiles && bits <= 4)) {
    const long long n16 = T * (d / 16), grid = (n16 + 255) / 256;
    if (grid > 0x7FFFFFFF) return set_error(GPTQ_ERR_INVALID_ARG, "too many tokens");
    widen_kernel<<<(unsigned)grid, 256, 0, s>>>(reinterpret_cast<const uint8_t*>(X), ldx, reinterpret_cast<uint16_t*>(ws), (int)d, n16);
    count_launch();
    if (gptq_status st = check_launch("widen_kernel")) return st;
    x = reinterpret_cast<const uint16_t*>(ws);
    ldx = d;
    x_dtype = GPTQ_BF16;
  }
  if (tiles)
    return linear_tiles_launch(qweight, scales, zeros, m, d, bits, group_size, x, x_dtype == GPTQ_E4M3, T, ldx, x_scale, bias, act,
                               mul, ldm, residual, ldr, Y, y_dtype, ldy, s);
  if (ids && plan_of(m, d, T, rank).N == 256) {
    float* z = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + adapter_workspace_bytes(m, d, bits, group_size, T, rank));
    if (gptq_status st = product_launch(Params{}, qweight, scales, zeros, m, d, bits, group_size, x, T, ldx, A, B, alpha, n_adapters, rank,
                                        ids, z, GPTQ_F32, m, ws, s))
      return st;
    EpiParams e{};
    e.x_scale = x_scale; e.bias = bias; e.act = act; e.mul = mul; e.residual = residual; e.ldm = ldm; e.ldr = ldr;
    e.Y = Y; e.ldy = ldy; e.m = (int)m; e.T = (int)T; e.y_bf16 = y_dtype == GPTQ_BF16;
    const unsigned gy = (unsigned)std::min<long long>(T, 32768);
    follow_kernel<<<dim3((unsigned)((m + 255) / 256), gy, (unsigned)((T + gy - 1) / gy)), 256, 0, s>>>(z, e);
    count_launch();
    return check_launch("follow_kernel");
  }
  EpiParams e{};
  e.x_scale = x_scale; e.bias = bias; e.act = act; e.mul = mul; e.residual = residual; e.ldm = ldm; e.ldr = ldr;
  e.wait_x = x != X;
  return product_launch(e, qweight, scales, zeros, m, d, bits, group_size, x, T, ldx, A, B, alpha, n_adapters, rank, ids, Y, y_dtype,
                        ldy, ws, s);
}

}  // namespace gptq
