// The gradient product (grad_tc.cu) of up to 8 tokens through an SC4 head, on warp MMAs.
//
// With few tokens the packed head is the work: V D / 2 bytes (N = 1, V = 151936, D = 4096: 311 of
// 341 MB).  A tcgen05 MMA takes its operands from shared memory, so every dequantised weight is
// written there and read back as FP16, and its 128 lanes are filled by one token or 128 alike: that
// kernel had its tensor pipe 79 % busy at N = 1 and took 122 us.  Here the head is the A operand of
// m16n8k16 and goes from its packed words into the fragments by register operations alone:
//  * k are vocabulary rows, m are columns, n tokens.  Lane (g, t) = (lane / 4, lane % 4) of a warp
//    holds rows t, t + 4, t + 8, t + 12 of the warp's 16 and the 8 columns of a packed word, chunk
//    i = g % 4 of block g / 4 of two 128-column blocks: 16 bytes per row, four words.  The low
//    bytes of two rows' words are put side by side; mask, subtract and multiply give two rows'
//    entries of one column as FP16, a register of A.  A word of four rows is four MMAs, a warp's
//    16 rows x 256 columns are 16.
//  * Sums stay in registers for the whole slab (64 a thread); at the end the warps' sums are added
//    through shared memory in their order and written to scratch as grad_tc_kernel does.
// Measured, cold caches: 89 us, 3.9 TB/s; four warps per scheduler issue in 63 % of the cycles, 2.7
// instructions per weight.  (A copy without the dequantisation took 20 us less: what is left then is
// the head's way through memory, 52 us, and the ends of the pipeline.)
// A unit of 128 rows x 256 columns (16 KB; its image: 256 bytes per token) comes by bulk copies into
// a ring, whose second block is placed 64 bytes further, so that 8 lanes read 128 bytes of all banks.
// The rank sums' tiles are 64 columns of the factor image, 16 KB per unit too.
#include "grad_common.cuh"

namespace archead {
namespace {

constexpr int kWarps = 8;  // 16 rows each: a unit
constexpr int kThreads = 32 * kWarps;
constexpr int kBlock1 = 8192 + 64;  // offset of the second block in a stage
constexpr int kImage = 2 * 8192 + 128;

constexpr int kTokens = 8;
constexpr int kStage = kImage + 256 * kTokens;
constexpr int kStages = 6;
constexpr int kSumRow = 257;  // floats per token of a warp's sums: tokens on different banks
constexpr size_t kSmem = (size_t)kStages * kStage + 16 * kStages + 128;
static_assert(kGradWarpCtas * (kSmem + 1024) <= 228 * 1024, "does not fit an SM");
static_assert(kWarps * kTokens * kSumRow * 4 <= kStages * kStage, "the warps' sums replace the ring");

__device__ __forceinline__ void mma_f16_16816(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t a) {
  unsigned short r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

// Two rows' entries of columns a and b, whose nibbles are the low byte's of each half (x), times
// their scales.  1024 + n and 64 + n are halves with the nibble in mantissa bits 0..3 and 4..7; its
// flipped top bit makes n = q + 8.  Both steps are exact.  (As fast as dequant_word's shifts and one
// fused multiply-add, which would need -24 c beside c in registers.)
__device__ __forceinline__ void entries(uint32_t x, __half2 c, uint32_t* a, uint32_t* b) {
  const __half2 lo = as_half2(and_xor(x, 0x000F000Fu, 0x64086408u)), hi = as_half2(and_xor(x, 0x00F000F0u, 0x54805480u));
  *a = h2_bits(__hmul2(__hsub2(lo, __float2half2_rn(1032.f)), c));
  *b = h2_bits(__hmul2(__hsub2(hi, __float2half2_rn(72.f)), c));
}

template <int CPC>
__global__ void __launch_bounds__(kThreads, kGradWarpCtas) grad_warp_kernel(const GradWarpParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStage);
  uint64_t* empty = full + kStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], kWarps);
    }
    tc::mbar_fence_init();
  }
  __syncthreads();
  const int nd = (int)((p.h.D + 255) >> 8);  // column tiles; the ranks' follow
  const int ntiles = nd + p.fcols / 64;
  const int slab = blockIdx.x / ntiles, tile = blockIdx.x - slab * ntiles;
  const bool rank = tile >= nd;
  const int64_t u0 = p.nunits * slab / p.slabs;
  const int count = (int)(p.nunits * (slab + 1) / p.slabs - u0);
  const bool two = rank || 256ll * tile + 128 < p.h.D;  // both 128-column blocks

  // Copies: the first round by one thread, the packed head before the wait, as it does not depend on
  // earlier kernels.  Then at unit k one warp in turn refills the slot of unit k - 2, which all warps
  // have mostly left by then.  (A warp of its own for this would cost a third of the registers; the
  // last warp to leave a slot, told by a counter, took 108 us, this 89.)
  const int64_t ublock = (p.h.D >> 7) << 13;  // bytes of a unit's rows in the packed head
  const int64_t ufact = (int64_t)p.fcols * 256;
  auto head_part = [&](int k) {
    unsigned char* dst = smem + (k % kStages) * kStage;
    uint64_t* bar = &full[k % kStages];
    tc::mbar_arrive_expect_tx(bar, (two ? 16384 : 8192) + 256 * kTokens);
    if (rank) return;
    const uint8_t* src = p.h.r_nib + (u0 + k) * ublock + ((int64_t)tile << 14);
    tc::bulk_g2s(dst, src, 8192, bar);
    if (two) tc::bulk_g2s(dst + kBlock1, src + 8192, 8192, bar);
  };
  auto other_part = [&](int k) {
    unsigned char* dst = smem + (k % kStages) * kStage;
    uint64_t* bar = &full[k % kStages];
    const char* img = p.img + (u0 + k) * 2 * (p.it * 128);
    tc::bulk_g2s(dst + kImage, img, 128 * kTokens, bar);
    tc::bulk_g2s(dst + kImage + 128 * kTokens, img + p.it * 128, 128 * kTokens, bar);
    if (!rank) return;
    const char* src = p.fimg + (u0 + k) * ufact + (tile - nd) * 4096;
    for (int q = 0; q < 4; ++q) tc::bulk_g2s(dst + 4096 * q, src + q * (ufact >> 2), 4096, bar);
  };
  const int ahead = count < kStages ? count : kStages;
  if (threadIdx.x == 0)
    for (int k = 0; k < ahead; ++k) head_part(k);
  grid_dependency_wait();  // cs and the images come from kernels before this one
  if (threadIdx.x == 0)
    for (int k = 0; k < ahead; ++k) other_part(k);
  int issued = threadIdx.x == 0 ? ahead - 1 : -1;  // the last unit that this thread has copied
  auto refill = [&](int k) {  // at unit k: the slot of unit k - 2
    if ((k & (kWarps - 1)) != warp) return true;
    const int next = k - 2 + kStages;
    if (k < 2 || next >= count) return true;
    const int st = (k - 2) % kStages;
    if (!__all_sync(0xffffffffu, tc::mbar_wait(&empty[st], (uint32_t)((k - 2) / kStages) & 1u, p.err))) return false;
    if (lane == 0) {
      tc::fence_proxy_async_smem();  // the warps' reads of the slot come before the copies
      head_part(next);
      other_part(next);
      issued = next;
    }
    __syncwarp();
    return true;
  };

  const int g = lane >> 2, t = lane & 3;
  float acc[4][4][4] = {};  // [word][MMA]
  const uint32_t base = tc::smem_u32(smem);
  // image: rows t + 4 j of this warp's 16, token g
  const int r0 = (16 * warp + t) & 63;
  const uint32_t b_at = base + kImage + (warp >> 2) * (128 * kTokens) + g * 128 + 2 * t;
  auto b_addr = [&](int j) {  // rows r0 + 4 j
    return b_at + (uint32_t)(((((r0 >> 3) + (j >> 1)) ^ g) & 7) << 4) + 8 * (j & 1);
  };
  bool ok = true;
  auto load_b = [&](uint32_t off, uint32_t b[2]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) b[q] = ld_shared_u16(b_addr(2 * q) + off) | ld_shared_u16(b_addr(2 * q + 1) + off) << 16;
  };
  if (rank) {
    // lane: chunk g (8 columns) of rows t + 4 j; MMA i takes columns 8 g + 2 i, + 1
    for (int k = 0; k < count; ++k) {
      const int st = k % kStages;
      if (!refill(k) || !__all_sync(0xffffffffu, tc::mbar_wait(&full[st], (uint32_t)(k / kStages) & 1u, p.err))) {
        ok = false;
        break;
      }
      const uint32_t off = st * kStage;
      uint32_t b[2], x[4][4];
      load_b(off, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kr = (16 * warp + t + 4 * j) & 31;
        const uint4 q = ld_shared16(base + off + (warp >> 1) * 4096 + (kr >> 3) * 1024 + (kr & 7) * 128 + (((g ^ kr) & 7) << 4));
        x[j][0] = q.x, x[j][1] = q.y, x[j][2] = q.z, x[j][3] = q.w;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty[st]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma_f16_16816(acc[0][i], __byte_perm(x[0][i], x[1][i], 0x5410), __byte_perm(x[0][i], x[1][i], 0x7632),
                      __byte_perm(x[2][i], x[3][i], 0x5410), __byte_perm(x[2][i], x[3][i], 0x7632), b[0], b[1]);
    }
  } else {
    // codes and row scales: lane l loads those of row l % 16, block l / 16, two units ahead
    const int64_t G = p.h.D >> p.g_shift;
    const int64_t v = u0 * 128 + 16 * warp + (lane & 15);
    const int64_t col = 256ll * tile + (two ? 128 * (lane >> 4) : 0);
    const uint8_t* code_at = p.h.r_code + v * G + (col >> p.g_shift);
    const uint32_t* cs_at = p.cs + v;
    uint32_t codes[2] = {}, cs[2] = {};
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (e < count) {
        codes[e] = load_codes<CPC>(code_at + e * 128 * G);
        cs[e] = load_word(cs_at + e * 128);
      }
    const uint32_t a_at = base + (g >> 2) * kBlock1 + ((g & 3) * 128 + 16 * warp + t) * 16;
    const int from = (lane >> 4) * 16 + t;  // the lane with row t of this lane's block
    // scales of rows t, t + 4 ([.][0]) and t + 8, t + 12 ([.][1]) in each window of 32 columns
    auto scales = [&](uint32_t code, uint32_t row, __half2 c[CPC][2]) {
#pragma unroll
      for (int n = 0; n < CPC; ++n) {
        const uint32_t own = h2_bits(code_half2(code, n, row));
        const uint32_t pair = __byte_perm(own, __shfl_xor_sync(0xffffffffu, own, 4), 0x5410);
        c[n][0] = as_half2(__shfl_sync(0xffffffffu, pair, from));
        c[n][1] = as_half2(__shfl_sync(0xffffffffu, pair, from + 8));
      }
    };
    code_at += 256 * G;
    cs_at += 256;
    __half2 c[CPC][2];
    scales(codes[0], cs[0], c);
    int st = 0;
    uint32_t phase = 0, off = 0;
    for (int k0 = 0; ok && k0 < count; k0 += 2) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = k0 + e;
        if (k >= count) break;
        if (!refill(k) || !__all_sync(0xffffffffu, tc::mbar_wait(&full[st], phase, p.err))) {
          ok = false;
          break;
        }
        uint32_t b[2];
        uint4 q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = ld_shared16(a_at + off + 64 * j);
        load_b(off, b);
        if (k + 2 < count) {
          codes[e] = load_codes<CPC>(code_at);
          cs[e] = load_word(cs_at);
          code_at += 128 * G;
          cs_at += 128;
        }
        __half2 cn[CPC][2];  // the next unit's, made beside this one's loads and MMAs
        scales(codes[1 - e], cs[1 - e], cn);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&empty[st]);
        off += kStage;
        if (++st == kStages) {
          st = 0;
          off = 0;
          phase ^= 1u;
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int n = CPC == 1 ? 0 : (CPC == 2 ? w >> 1 : w);
          const __half2 ca = c[n][0], cb = c[n][1];
          uint32_t x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = w == 0 ? q[j].x : (w == 1 ? q[j].y : (w == 2 ? q[j].z : q[j].w));
          uint32_t a0[4], a1[4], a2[4], a3[4];
          // bytes 0 and 1 of a word: its even columns' nibbles 0, 1 and 2, 3; bytes 2 and 3: the odd ones'
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t s0 = h ? 0x0501 : 0x0400, s1 = h ? 0x0703 : 0x0602;
            entries(__byte_perm(x[0], x[1], s0), ca, &a0[2 * h], &a0[2 * h + 1]);
            entries(__byte_perm(x[0], x[1], s1), ca, &a1[2 * h], &a1[2 * h + 1]);
            entries(__byte_perm(x[2], x[3], s0), cb, &a2[2 * h], &a2[2 * h + 1]);
            entries(__byte_perm(x[2], x[3], s1), cb, &a3[2 * h], &a3[2 * h + 1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
mma_f16_16816(acc[w][i], a0[i], a1[i], a2[i], a3[i], b[0], b[1]);
        }
#pragma unroll
        for (int n = 0; n < CPC; ++n) c[n][0] = cn[n][0], c[n][1] = cn[n][1];
      }
    }
  }

  // ---- the warps' sums, through the ring's memory ----
  if (!__syncthreads_and(ok)) {
    // no copy may be in flight at the end (on the other way every unit has been waited for)
    for (int k = issued; k >= 0 && k > issued - kStages; --k)
      tc::mbar_wait(&full[k % kStages], (uint32_t)(k / kStages) & 1u, p.err);
    return;
  }
  float* sums = reinterpret_cast<float*>(smem);
  const int words = rank ? 1 : 4;
#pragma unroll
  for (int w = 0; w < 4; ++w)
    if (w < words)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = (rank ? 8 * g : 128 * (g >> 2) + 32 * w + 8 * (g & 3)) + 2 * i + (e >> 1);
          sums[(warp * kTokens + 2 * t + (e & 1)) * kSumRow + col] = acc[w][i][e];
        }
  __syncthreads();
  const int RR = p.h.r_c + p.h.r_r;
  const int col = threadIdx.x;
  const int live = rank ? min(64, RR - 64 * (tile - nd)) : (two ? 256 : 128);
  if (col >= live) return;
  float* dst = p.part + (int64_t)slab * p.n * p.dp + (rank ? p.h.D + 64 * (tile - nd) : 256ll * tile) + col;
#pragma unroll 1
  for (int n = 0; n < p.n; ++n) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[(w * kTokens + n) * kSumRow + col];
    dst[n * p.dp] = s;
  }
}

template <int CPC>
cudaError_t launch_groups(const GradWarpParams& p, cudaStream_t st) {
  auto kern = grad_warp_kernel<CPC>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((p.h.D + 255) / 256 + p.fcols / 64) * p.slabs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_grad_warp(const GradWarpParams& p, cudaStream_t st) {
  if (p.h.g == 32) return launch_groups<4>(p, st);
  if (p.h.g == 64) return launch_groups<2>(p, st);
  return launch_groups<1>(p, st);
}

}  // namespace archead
