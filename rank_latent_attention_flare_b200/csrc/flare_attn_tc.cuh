// Pieces shared by the tensor-core attention kernels (forward and backward):
// operand tiles, their descriptors and tensor maps.
#pragma once

#include <cudaTypedefs.h>

#include "flare_attn.cuh"
#include "tc_primitives.cuh"

namespace flare {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace attn {

using namespace tc;

constexpr int kMinSmemBytes = 120 * 1024;   // keeps one CTA (and its TMEM) per SM

// A tile of 128 rows of DP bf16 elements in shared memory: rows of 128 bytes
// (64 elements) under the 128-byte swizzle, two such blocks side by side for
// DP = 128; rows of 64 bytes under the 64-byte swizzle for DP = 32.
template <int DP>
struct Tile {
  static constexpr int RB = DP < 64 ? 2 * DP : 128;
  static constexpr int BLOCKS = DP == 128 ? 2 : 1;
  static constexpr int BLOCK = 128 * RB;
  static constexpr int BYTES = BLOCK * BLOCKS;
  static constexpr uint32_t SW = RB == 128 ? 2u : 4u;
  // address-field step of K step kk (16 elements of D) of a K-major operand
  static __device__ __forceinline__ constexpr uint32_t kstep(int kk) {
    return RB == 128 ? ((kk >> 2) * BLOCK + (kk & 3) * 32) >> 4 : (kk * 32) >> 4;
  }
  // rows as the MMA's M or N, D as its K
  static __device__ __forceinline__ uint64_t k_major(uint32_t addr) {
    return smem_desc(addr, 16, 8 * RB, SW);
  }
  // D as the MMA's N, rows as its K: 16 rows per K step
  static __device__ __forceinline__ uint64_t mn_major(uint32_t addr) {
    return smem_desc(addr, BLOCK, 8 * RB, SW);
  }
  static constexpr uint32_t MN_STEP = (16 * RB) >> 4;
};

// Loads rows [row, row + box) of head h of batch b (all column blocks).
template <int DP>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar,
                                          int row, int h, int b) {
#pragma unroll
  for (int k = 0; k < Tile<DP>::BLOCKS; ++k)
    tma_load_4d(dst + k * Tile<DP>::BLOCK, map, bar, 64 * k, row, h, b);
}

// One arrival for the whole warp, once all its lanes are here.  Predicated,
// so that the warp stays converged for the collective instructions after it.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(threadIdx.x & 31u)
      : "memory");
}

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return (uint8_t*)(((uintptr_t)p + 1023) & ~(uintptr_t)1023);
}

// Tensor map over a [B,H,N,D] bf16 tensor with strides t (dimensions
// {D, N, H, B}; a zero stride makes a dimension of one entry), boxes of
// `rows` rows of `heads` heads and min(DP, 64) columns, swizzled as Tile<DP>.
inline cudaError_t attn_map(CUtensorMap* m, const void* base, const Tok& t, int64_t B, int64_t H,
                            int64_t N, int64_t D, int dp, int rows, int heads) {
  auto enc = tensor_map_encoder();
  if (!enc) {
    note_error("cuTensorMapEncodeTiled entry point unavailable");
    return cudaErrorNotSupported;
  }
  const cuuint64_t any = (cuuint64_t)D * 2;   // for a dimension of one entry (not used)
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)(t.sh ? H : 1),
                        (cuuint64_t)(t.sb ? B : 1)};
  cuuint64_t strides[3] = {N > 1 ? (cuuint64_t)t.sn * 2 : any,
                           dims[2] > 1 ? (cuuint64_t)t.sh * 2 : any,
                           dims[3] > 1 ? (cuuint64_t)t.sb * 2 : any};
  cuuint32_t box[4] = {(cuuint32_t)(dp < 64 ? dp : 64), (cuuint32_t)rows, (cuuint32_t)heads, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   dp < 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    note_error("cuTensorMapEncodeTiled failed (CUresult %d): attention map D=%lld N=%lld H=%lld "
               "B=%lld strides %lld/%lld/%lld box %dx%d",
               (int)r, (long long)D, (long long)N, (long long)H, (long long)B, (long long)t.sb,
               (long long)t.sh, (long long)t.sn, rows, heads);
    return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

// Waits for two 64-column loads in flight, naming every register they write.
__device__ __forceinline__ void tmem_wait_ld_dep128(uint32_t (&a)[64], uint32_t (&b)[64]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]),
                 "+r"(a[7]), "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]),
                 "+r"(a[13]), "+r"(a[14]), "+r"(a[15]), "+r"(a[16]), "+r"(a[17]), "+r"(a[18]),
                 "+r"(a[19]), "+r"(a[20]), "+r"(a[21]), "+r"(a[22]), "+r"(a[23]), "+r"(a[24]),
                 "+r"(a[25]), "+r"(a[26]), "+r"(a[27]), "+r"(a[28]), "+r"(a[29]), "+r"(a[30]),
                 "+r"(a[31]), "+r"(a[32]), "+r"(a[33]), "+r"(a[34]), "+r"(a[35]), "+r"(a[36]),
                 "+r"(a[37]), "+r"(a[38]), "+r"(a[39]), "+r"(a[40]), "+r"(a[41]), "+r"(a[42]),
                 "+r"(a[43]), "+r"(a[44]), "+r"(a[45]), "+r"(a[46]), "+r"(a[47]), "+r"(a[48]),
                 "+r"(a[49]), "+r"(a[50]), "+r"(a[51]), "+r"(a[52]), "+r"(a[53]), "+r"(a[54]),
                 "+r"(a[55]), "+r"(a[56]), "+r"(a[57]), "+r"(a[58]), "+r"(a[59]), "+r"(a[60]),
                 "+r"(a[61]), "+r"(a[62]), "+r"(a[63]), "+r"(b[0]), "+r"(b[1]), "+r"(b[2]),
                 "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7]), "+r"(b[8]), "+r"(b[9]),
                 "+r"(b[10]), "+r"(b[11]), "+r"(b[12]), "+r"(b[13]), "+r"(b[14]), "+r"(b[15]),
                 "+r"(b[16]), "+r"(b[17]), "+r"(b[18]), "+r"(b[19]), "+r"(b[20]), "+r"(b[21]),
                 "+r"(b[22]), "+r"(b[23]), "+r"(b[24]), "+r"(b[25]), "+r"(b[26]), "+r"(b[27]),
                 "+r"(b[28]), "+r"(b[29]), "+r"(b[30]), "+r"(b[31]), "+r"(b[32]), "+r"(b[33]),
                 "+r"(b[34]), "+r"(b[35]), "+r"(b[36]), "+r"(b[37]), "+r"(b[38]), "+r"(b[39]),
                 "+r"(b[40]), "+r"(b[41]), "+r"(b[42]), "+r"(b[43]), "+r"(b[44]), "+r"(b[45]),
                 "+r"(b[46]), "+r"(b[47]), "+r"(b[48]), "+r"(b[49]), "+r"(b[50]), "+r"(b[51]),
                 "+r"(b[52]), "+r"(b[53]), "+r"(b[54]), "+r"(b[55]), "+r"(b[56]), "+r"(b[57]),
                 "+r"(b[58]), "+r"(b[59]), "+r"(b[60]), "+r"(b[61]), "+r"(b[62]), "+r"(b[63])
               :
               : "memory");
}

// Raw logits outside columns [lo, hi] become -inf.
template <int N>
__device__ __forceinline__ void mask_cols(uint32_t (&a)[N], int col0, int lo, int hi) {
#pragma unroll
  for (int t = 0; t < N; ++t)
    if (col0 + t < lo || col0 + t > hi) a[t] = 0xff800000u;
}

// Three-input maximum that is NaN when one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Max of 64 values folded into four independent accumulators (NaN: one was).
__device__ __forceinline__ void max_fold64(const uint32_t (&a)[64], float (&m)[4]) {
#pragma unroll
  for (int t = 0; t < 64; t += 8) {
    m[0] = max3_nan(m[0], __uint_as_float(a[t + 0]), __uint_as_float(a[t + 1]));
    m[1] = max3_nan(m[1], __uint_as_float(a[t + 2]), __uint_as_float(a[t + 3]));
    m[2] = max3_nan(m[2], __uint_as_float(a[t + 4]), __uint_as_float(a[t + 5]));
    m[3] = max3_nan(m[3], __uint_as_float(a[t + 6]), __uint_as_float(a[t + 7]));
  }
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Writes 32 consecutive fp32 values times f as bf16 to p[0..32), the columns
// below D only (D and col0 are multiples of 8, rows 16-byte aligned); with
// `low` also what the rounding left over, rounded to bf16.
__device__ __forceinline__ void store_bf16x32(__nv_bfloat16* p, const uint32_t (&o)[32], float f,
                                              int col0, int D, __nv_bfloat16* low = nullptr) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (col0 + 8 * g >= D) break;
    uint32_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = pack_bf16(__uint_as_float(o[8 * g + 2 * k]) * f,
                       __uint_as_float(o[8 * g + 2 * k + 1]) * f);
    *reinterpret_cast<uint4*>(p + 8 * g) = make_uint4(v[0], v[1], v[2], v[3]);
    if (low == nullptr) continue;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = pack_bf16(fmaf(__uint_as_float(o[8 * g + 2 * k]), f, -bf_lo(v[k])),
                       fmaf(__uint_as_float(o[8 * g + 2 * k + 1]), f, -bf_hi(v[k])));
    *reinterpret_cast<uint4*>(low + 8 * g) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

}  // namespace attn
}  // namespace flare
