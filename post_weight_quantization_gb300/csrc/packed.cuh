// What the products of packed layers share: codes to numbers in registers, the reads of staged codes,
// issuing on the tensor core by one lane of a converged warp, paired fp32 arithmetic, activations.
#pragma once

#include <cudaTypedefs.h>

#include "elem.cuh"

namespace gptq {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();   // tc_gemm.cu

namespace adp {

constexpr int BM = 128, KB = 128;                        // rows of a tile, columns of a block of codes

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
// c * 2^-133 (a bf16 pair of small integers' bits) to (c - zero) * 2^-6; nz is the pair -zero * 2^-6
__device__ __forceinline__ uint32_t to_int(uint32_t c, uint32_t nz) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(c), "r"(0x7F007F00u), "r"(nz));
  return d;
}
__device__ __forceinline__ uint32_t neg_zero(float z) {
  return (__float_as_uint(-z * 0.015625f) >> 16) * 0x00010001u;      // an integer below 256: exact in bf16
}

// 32 codes (BITS words) as 16 bf16 pairs of (code - zero) * 2^-6 in the columns' order.
template <int BITS>
__device__ __forceinline__ void unpack32(const uint32_t* w, uint32_t nz, uint32_t (&o)[16]) {
  if constexpr (BITS == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t e = w[j] & 0x0F0F0F0Fu, d = (w[j] >> 4) & 0x0F0F0F0Fu;
#pragma unroll
      for (int i = 0; i < 4; ++i)           // bytes i of both; a selector's top bit repeats a byte's sign bit: 0
        o[4 * j + i] = to_int(prmt(e, d, (uint32_t)(i | ((8 + i) << 4) | ((4 + i) << 8) | ((12 + i) << 12))), nz);
    }
  } else if constexpr (BITS == 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      o[2 * j] = to_int(prmt(w[j], 0u, 0x4140u), nz);
      o[2 * j + 1] = to_int(prmt(w[j], 0u, 0x4342u), nz);
    }
  } else if constexpr (BITS == 2) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = (w[j] >> (2 * k)) & 0x03030303u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t sel = (uint32_t)(i | ((8 + i) << 4) | ((4 + i) << 8) | ((12 + i) << 12));
        o[8 * j + 2 * i] = to_int(prmt(c[0], c[1], sel), nz);
        o[8 * j + 2 * i + 1] = to_int(prmt(c[2], c[3], sel), nz);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int b = 6 * i, k = b >> 5, sh = b & 31;
      const uint32_t s = k < 2 ? __funnelshift_r(w[k], w[k + 1], sh) : w[2] >> sh;
      o[i] = to_int((s & 7u) | ((s << 13) & 0x00070000u), nz);
    }
  }
}

template <int N>
__device__ __forceinline__ void load_words(const uint32_t* p, uint32_t* w) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + i));
      w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(p + i);
  }
}

// 16 bytes (piece i) of row r from a stage of packed codes. Rows are swizzled as their length asks,
// so that eight lanes reading eight rows meet no bank twice (3 bits: 48-byte rows need none).
template <int BITS>
__device__ __forceinline__ void lds_piece(uint32_t stage, int r, int i, uint32_t* w) {
  const int at = BITS == 8 ? i ^ (r & 7) : BITS == 4 ? i ^ ((r >> 1) & 3) : BITS == 2 ? i ^ ((r >> 2) & 1) : i;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(stage + r * (16 * BITS) + at * 16));
}

__device__ __forceinline__ void umma_commit_by(uint64_t* bar, uint32_t leader) {
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

// Pairs of fp32 in one 64-bit register pair, two operations an instruction.
__device__ __forceinline__ uint64_t pack2u(uint32_t lo, uint32_t hi) { return (uint64_t)lo | ((uint64_t)hi << 32); }
__device__ __forceinline__ uint64_t pack2(float lo, float hi) { return pack2u(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float half2f(uint64_t v, int i) { return __uint_as_float((uint32_t)(i ? v >> 32 : v)); }
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

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r) {
  if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  }
}

// A value for each of many a thread, so by the fast exponential and quotient, which err by 2 + 1.2 y and 2 units of fp32's last
// place, y the exponent's size. Counted in 2^-23 of |act(z)|: silu 5 + 1.2 |z|; gelu_tanh 5 + 4.2 y, y = 1.6 |z| (1 + 0.045 z^2), whose
// exponent is itself off by 3 y; gelu (erfcf by 4, its argument's rounding by z^2 + |z|) 5 + z^2 + |z|; for positive z all of them 5
// at most, as the exponential is the smaller part of 1 + e there. silu and gelu_tanh are 0 where their divisor passes 2^126.
// bf16 outputs are rounded by 2^15 of these units; in fp32 outputs of large negative z, themselves next to 0, the errors are seen.
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case GPTQ_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case GPTQ_ACT_SILU: return __fdividef(z, 1.0f + __expf(-z));
    case GPTQ_ACT_GELU: return 0.5f * z * erfcf(-0.707106781f * z);
    case GPTQ_ACT_GELU_TANH:                               // 1 + tanh(y) = 2 / (1 + e^(-2 y))
      return __fdividef(z, 1.0f + __expf(-1.59576912f * fmaf(0.044715f * z * z, z, z)));
    default: return z;
  }
}
__device__ __forceinline__ float read_y(const void* p, long long at, long long bf16) {
  return bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[at]) : reinterpret_cast<const float*>(p)[at];
}

// The packed rows as bytes, a block's 16 * bits of 128 rows a box. False where TMA cannot take them
// (rows that are no multiple of 16 bytes: 2 bits with d % 64, 3 bits with d % 128, or a base that
// is not 16-byte aligned): the unpacking warps then read their rows from global memory.
inline bool make_code_map(CUtensorMap* m, const void* base, long long rows, long long row_bytes, int bits) {
  auto enc = tensor_map_encoder();
  if (!enc || row_bytes % 16 || reinterpret_cast<uintptr_t>(base) % 16) return false;
  cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  cuuint32_t box[2] = {(cuuint32_t)(16 * bits), BM};
  cuuint32_t es[2] = {1, 1};
  const CUtensorMapSwizzle sw = bits == 8 ? CU_TENSOR_MAP_SWIZZLE_128B
                                : bits == 4 ? CU_TENSOR_MAP_SWIZZLE_64B
                                            : bits == 2 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_NONE;
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace adp
}  // namespace gptq
