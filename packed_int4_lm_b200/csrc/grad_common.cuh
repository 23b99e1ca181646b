// Shared by the kernels of the gradient product (grad_tc.cu) and those that write its operand
// image: the per-row scale, the image's layout, and pieces of their tcgen05 pipelines.
#pragma once

#include "tc_common.cuh"

namespace archead {

// Row scale of the gradient product.  The product's operands are FP16, so vocabulary row v is
// split into a scale S'_v, folded into dY, and entries that FP16 holds: the residual q c 2^-k,
// exact for k <= 24, and the factor entries a / S', |a| / S' < 2^14.  With M = 128 max(|sAc|,
// |sAw|) bounding the factor entries, S' = S 2^k with k = ilogb(M) - ilogb(S) - 13, at least -3
// (the dequantisation's addend 24 c 2^-k must stay finite).  From k = 25 on (M >= 2^38 S) the scales
// c 2^-k keep fewer bits, as in the logits' tcgen05 kernel, and none from 33 on.  Where S is 0, or k would
// pass 40, the residual is dropped and S' comes from M alone; a row without either has S' = 0.  A factor
// entry is one FP16 value (11 bits, as dY; the result keeps 8), of fewer bits below 2^-14 S'.  The rule
// looks at the left factors alone, so it relies on right factors that are not tiny or huge; the header
// states the limits.
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

// The product of up to 8 tokens through an SC4 head (grad_warp.cu): the FP32 sums of each slab of the
// vocabulary, [slab][n][dp], columns 0 .. D - 1 and then the ranks.
struct GradWarpParams {
  archead_head h;
  const char* img;  // image tiles of `it` tokens
  const uint32_t* cs;  // per row 2^(8 - k), FP16x2
  const char* fimg;  // factor image: per 32 rows, fcols x 64 bytes
  float* part;
  int64_t n, dp, nunits;
  int it, fcols, slabs, g_shift;
  unsigned* err;
};
constexpr int kGradWarpCtas = 2;  // per SM
cudaError_t launch_grad_warp(const GradWarpParams& p, cudaStream_t st);

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

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D[tmem] (+)= A[smem] * B[smem]^T, one M=128 x N x K=16 step, issued by one thread.
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// mbar_wait for a wait of many microseconds: sleeps between polls, which would otherwise take
// issue slots and power from the warps that work.
__device__ __forceinline__ bool mbar_wait_long(uint64_t* bar, uint32_t parity, unsigned* err) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!tc::mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > (1ll << 31)) {
      atomicOr(err, kErrTimeout);
      return false;
    }
    __nanosleep(200);
  }
  return true;
}

// The code bytes (CPC of them) of one vocabulary row for one block of 128 columns, and its word of
// the row table.  Volatile: issued here, an iteration before their use (the compiler would move
// plain loads down to it, where they cost a round trip to memory per unit).
template <int CPC>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* c) {
  uint32_t r;
  if (CPC == 1) asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(r) : "l"(c));
  else if (CPC == 2) asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(r) : "l"(c));  // (zero-extended)
  else asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(r) : "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t load_word(const uint32_t* c) {
  uint32_t r;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(r) : "l"(c));
  return r;
}
// Code e of them times 2^-k, twice in FP16 (exact for k <= 24): 4 + c 2^-8 is a half with the byte c in
// its low mantissa bits, and cs = 2^(8 - k) is an FP16 number up to k = 32.
__device__ __forceinline__ __half2 code_half2(uint32_t codes, int e, uint32_t cs) {
  const uint32_t r = __byte_perm(codes, 0x44444444u, 0x4040u + 0x0101u * e);
  return __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&r), __float2half2_rn(4.f)),
                 *reinterpret_cast<const __half2*>(&cs));
}

}  // namespace archead
