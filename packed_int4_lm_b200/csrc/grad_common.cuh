// Shared by the kernels of the gradient product (grad_tc.cu) and those that write its operand
// image: the per-row scale and the image's layout.
#pragma once

#include "archead_internal.cuh"

namespace archead {

// Row scale of the gradient product.  The product's operands are FP16, so vocabulary row v is
// split into a scale S'_v, folded into dY, and entries that FP16 holds: the residual q c 2^-k,
// exact for k <= 24, and the factor entries a / S', |a| / S' < 2^14.  With M = 128 max(|sAc|,
// |sAw|) bounding the factor entries, S' = S 2^k with k = ilogb(M) - ilogb(S) - 13, at least -3
// (the dequantisation's addend 24 c 2^-k must stay finite).  Where S is 0, or k would pass 40
// (the residual is then under 2^-45 of the factors' bound), the residual is dropped and S' comes
// from M alone; a row without either has S' = 0.
struct GradRow {
  float sp;  // S'
  float cs;  // 2^-k, 0 without a residual
};
__host__ __device__ __forceinline__ GradRow grad_row(float S, float sac, float saw) {
  const float M = 128.f * fmaxf(fabsf(sac), fabsf(saw));
  GradRow r = {S, S != 0.f ? 1.f : 0.f};
  if (M > 0.f) {
    int k = S != 0.f ? ilogbf(M) - ilogbf(S) - 13 : 41;
    if (k > 40) {
      r.sp = ldexpf(1.f, ilogbf(M) - 13);
      r.cs = 0.f;
    } else {
      if (k < -3) k = -3;
      r.sp = ldexpf(S, k);
      r.cs = ldexpf(1.f, -k);
    }
  }
  return r;
}

// Image of dY, the product's B operand: per token tile of nt rows and 64 vocabulary rows
// (half-unit hb) a block of nt x 128 bytes, token nn's 64 FP16 values in one 128-byte row whose
// 16-byte chunk c is stored at c ^ (nn % 8) (the K-major 128-byte swizzle).  Byte offset of the
// value of vocabulary row 64 hb + r:
__host__ __device__ __forceinline__ int64_t grad_image_offset(int64_t tt, int64_t hb, int64_t nhb,
                                                              int nt, int nn, int r) {
  return ((tt * nhb + hb) * nt + nn) * 128 + ((((r >> 3) ^ nn) & 7) << 4) + 2 * (r & 7);
}

// Power of two 2^e, as two factors that stay inside FP32's range for |e| <= 250.
__device__ __forceinline__ void pow2_pair(int e, float* a, float* b) {
  const int h = e / 2;
  *a = __int_as_float((h + 127) << 23);
  *b = __int_as_float((e - h + 127) << 23);
}

// Two signed bytes of w (its bytes sel picks, offset by 128) as exact FP16: the half 1024 + 128 + b
// has the low mantissa byte b ^ 0x80.
__device__ __forceinline__ __half2 bytes_to_half2(uint32_t w_flipped, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(w_flipped), "r"(0x64646464u), "r"(sel));
  return __hsub2(*reinterpret_cast<__half2*>(&r), __float2half2_rn(1152.f));
}

}  // namespace archead
