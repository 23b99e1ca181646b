// Logits of large batches straight into the softmax gradient's FP16 image (grad_common.cuh):
//
//   img[n, v] = exp(Y[n, v] - lse[n]) 2^f_n S'_v 2^-es,   Y = S'_v 2^e_n (sum_d h'[n, d] w[v, d] + ...)
//
// the same sums as the logits kernel of residual_tc.cu (residual columns q c 2^-k, rank columns as
// FP16 pieces), with tiles of 256 tokens x 256 vocabulary rows: a dequantised weight serves 256
// tokens there against 128, so half the dequantisation, and the tensor cores read 12 KB of shared
// memory per 128 x 256 x 16 step (that and the stores and copies, about 160 KB per step of 64
// columns, are what bounds it: 1300 cycles against the MMAs' 1024).  N = 4096 on the 151936 x 4096
// head: 3.67 ms against 4.28 ms (1405 against 1204 TFLOP/s).
//
// Persistent, one CTA per SM.  The tokens are the accumulators' lanes (A: the blocked FP16 image of
// H, 128 tokens each, two accumulators), the vocabulary rows their columns (B, K-major).
//  * warps 0-15: lane = vocabulary row of a 32-row group; packed chunks from global memory into
//    registers a unit (128 columns) ahead, exact FP16 entries into the two W stages of the unit;
//    then the rank columns from the INT8 factors;
//  * warps 16-23: epilogue, four per accumulator, lane = token: one exp2 per entry with all scales
//    in its exponent, eight entries per 16-byte store;
//  * warp 24: bulk copies of the H image; warps 25, 26: MMA issuers, an accumulator each.
// Targets' entries are set afterwards (grad_targets).  Every wait is bounded.
#include "grad_common.cuh"

namespace archead {
namespace {

constexpr int kSmThreads = 32 * 27;
constexpr int kStage = 256 * 128;   // W stage: 256 rows x 64 columns FP16
constexpr int kHStage = 128 * 128;  // image stage: 128 tokens x 64 columns FP16
constexpr int kSW = 3, kSH = 8;     // 96 KB and 128 KB
constexpr size_t kSmSmem = (size_t)kSW * kStage + kSH * kHStage + 256 * 8 + 512;
static_assert(kSmSmem <= 227 * 1024, "does not fit an SM");

struct SoftmaxParams {
  archead_head h;
  const char* himg;  // [token tile of 128][nkb + nrb blocks][two halves][128 x 128 bytes]
  const float* tsc;
  const float* sp;
  const uint32_t* cs;
  TcImage out;  // nt = 128
  int64_t n;
  int64_t nvt;   // 128-row tiles of the vocabulary
  int64_t items;
  int ntile;     // token tiles of 128
  int npair;     // pairs of them
  int band;      // pairs whose H image stays in L2 together
  int nkb, nrb, g_shift, a_words;
  unsigned* err;
};

struct SmItem {
  int64_t vt;  // pair of 128-row tiles
  int tp, m;   // token pair, its tiles
};
__device__ __forceinline__ bool sm_item(const SoftmaxParams& p, int64_t k, SmItem& it) {
  const int64_t i = blockIdx.x + k * gridDim.x;
  if (i >= p.items) return false;
  // bands of token pairs; inside one the pair varies fastest, so that CTAs side by side share
  // vocabulary rows
  const int64_t nv2 = (p.nvt + 1) >> 1, per = nv2 * p.band, b = i / per, local = i - b * per;
  const int64_t t0 = b * p.band, nb = p.npair - t0 < p.band ? p.npair - t0 : p.band;
  it.vt = local / nb;
  it.tp = (int)(t0 + (local - it.vt * nb));
  it.m = p.ntile - 2 * it.tp < 2 ? 1 : 2;
  return true;
}

__device__ __forceinline__ uint32_t sm_factor_word(const SoftmaxParams& p, int64_t v, int j) {
  const int rc = p.h.r_c, rr = p.h.r_r;
  if (p.a_words) {
    if (j < rc) return __ldg(reinterpret_cast<const uint32_t*>(p.h.Ac + v * rc + j));
    if (j < rc + rr) return __ldg(reinterpret_cast<const uint32_t*>(p.h.Aw + v * rr + (j - rc)));
    return 0u;
  }
  uint32_t w = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int jj = j + u;
    int8_t b = 0;
    if (jj < rc) b = __ldg(p.h.Ac + v * rc + jj);
    else if (jj < rc + rr) b = __ldg(p.h.Aw + v * rr + (jj - rc));
    w |= (uint32_t)(uint8_t)b << (8 * u);
  }
  return w;
}

template <int CPC>
__global__ void __launch_bounds__(kSmThreads, 1) softmax_tc_kernel(const SoftmaxParams p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* Ws = smem;
  unsigned char* Hs = Ws + kSW * kStage;
  float2* rows_s = reinterpret_cast<float2*>(Hs + kSH * kHStage);  // S'_v, log2 |S'_v|
  uint64_t* w_full = reinterpret_cast<uint64_t*>(rows_s + 256);
  uint64_t* w_empty = w_full + kSW;
  uint64_t* h_full = w_empty + kSW;
  uint64_t* h_empty = h_full + kSH;
  uint64_t* acc_full = h_empty + kSH;   // [2]
  uint64_t* acc_empty = acc_full + 2;   // [2]
  uint64_t* mma_done = acc_empty + 2;   // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSW; ++i) {
      tc::mbar_init(&w_full[i], 16);
      tc::mbar_init(&w_empty[i], 2);
    }
    for (int i = 0; i < kSH; ++i) {
      tc::mbar_init(&h_full[i], 1);
      tc::mbar_init(&h_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&acc_full[i], 1);
      tc::mbar_init(&acc_empty[i], 128);
      tc::mbar_init(&mma_done[i], 1);
    }
    tc::mbar_fence_init();
  }
  if (warp == 25) tc::tmem_alloc(tmem_slot, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  const int nkbt = p.nkb + p.nrb;
  SmItem it;

  if (warp < 16) {
    // ---- dequantisation ----
    // Rows 32 rg .. + 31 of the tile pair, half of the block's 16-byte chunks; a unit of 128 columns
    // is two W stages (windows 0, 1 and 2, 3), all sixteen warps fill both.
    const int rg = warp & 7, ch = warp >> 3, r = 32 * rg + lane;
    const uint32_t w_addr = tc::smem_u32(Ws) + (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((r & 7) << 4));
    int slot = 0;
    uint32_t wp = 1;  // parity of the slot's last release (the first use waits for none)
    bool ok = true;
    grid_dependency_wait();  // the row tables come from a kernel before this one
    const int64_t G = p.h.D >> p.g_shift;
    // o: the chunks of one stage, in order; the entries are in registers before the wait
    auto put = [&](const uint32_t (&o)[4][4], const int (&chunk)[4], bool ready) -> bool {
      if (!__all_sync(0xffffffffu, ready) && !__all_sync(0xffffffffu, tc::mbar_wait(&w_empty[slot], wp, p.err)))
        return false;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        st_shared16((w_addr ^ (uint32_t)(chunk[c] << 4)) + slot * kStage, o[c][0], o[c][1], o[c][2], o[c][3]);
      tc::fence_proxy_async_smem();  // the MMA reads the stage through the async proxy
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&w_full[slot]);
      if (++slot == kSW) {
        slot = 0;
        wp ^= 1u;
      }
      return true;
    };
    for (int64_t i = 0; ok && sm_item(p, i, it); ++i) {
      const int64_t T = 2 * it.vt + (rg >> 2);  // (warp-uniform; the pair's second tile may not exist)
      const bool work = T < p.nvt;
      const int64_t Tc = work ? T : T - 1;
      const int s = 32 * (rg & 3) + lane;
      const int64_t v = 128 * Tc + s;
      const uint8_t* p_at = p.h.r_nib + ((Tc * p.nkb) << 13) + s * 16 + 2 * ch * 2048;
      const uint8_t* code_at = p.h.r_code + v * G;
      const uint32_t cs = load_word(p.cs + v);
      uint32_t codes = load_codes<CPC>(code_at);
      uint4 q[2] = {ldg_stream(p_at), ldg_stream(p_at + 2048)};
      for (int kb = 0; kb < p.nkb; ++kb) {
        const bool more = kb + 1 < p.nkb;
        const bool ready = tc::mbar_test(&w_empty[slot], wp);
        const uint32_t now = codes;
        if (more) codes = load_codes<CPC>(code_at + (((kb + 1) * 128) >> p.g_shift));
        uint32_t o[2][4][4];
#pragma unroll
        for (int wn = 0; wn < 4; ++wn) {
          const __half2 c2 = code_half2(now, CPC == 1 ? 0 : (CPC == 2 ? wn >> 1 : wn), cs);
          const __half2 nc24 = __hmul2(c2, __float2half2_rn(-24.f));
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 x = q[c];
            const uint32_t word = wn == 0 ? x.x : (wn == 1 ? x.y : (wn == 2 ? x.z : x.w));
            __half2 e[4];
            dequant_word(word, c2, nc24, e);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[wn >> 1][2 * (wn & 1) + c][j] = h2_bits(e[j]);
          }
        }
        if (more) {
          p_at += 8192;
          q[0] = ldg_stream(p_at);
          q[1] = ldg_stream(p_at + 2048);
        }
        const int chunk[4] = {2 * ch, 2 * ch + 1, 4 + 2 * ch, 5 + 2 * ch};
        if (!put(o[0], chunk, ready) || !put(o[1], chunk, false)) {
          ok = false;
          break;
        }
      }
      if (!ok) break;
      // rank columns: factor index j takes (x1, x1, x2, x2), x = fl32(A[v, j] s_v) / S'; a stage
      // holds 16 indices, this warp's chunks 4 ch .. + 3 eight of them
      const bool live = work && v < p.h.V;
      const float sac = live && p.h.r_c ? __ldg(p.h.sAc + v) : 0.f, saw = live && p.h.r_r ? __ldg(p.h.sAw + v) : 0.f;
      const float sp = __ldg(p.sp + v), rcp = sp != 0.f ? 1.f / sp : 0.f;
      for (int st = 0; st < 2 * p.nrb; ++st) {
        const int j0 = 16 * st + 8 * ch;
        uint32_t o[4][4];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t fw = live ? sm_factor_word(p, v, j0 + 4 * w) : 0u;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float x = __fmul_rn((float)(int8_t)((fw >> (8 * u)) & 0xFFu), j0 + 4 * w + u < p.h.r_c ? sac : saw) * rcp;
            const __half x1 = __float2half_rn(x), x2 = __float2half_rn(x - __half2float(x1));
            o[2 * w + (u >> 1)][2 * (u & 1)] = h2_bits(__half2half2(x1));
            o[2 * w + (u >> 1)][2 * (u & 1) + 1] = h2_bits(__half2half2(x2));
          }
        }
        const int chunk[4] = {4 * ch, 4 * ch + 1, 4 * ch + 2, 4 * ch + 3};
        if (!put(o, chunk, false)) {
          ok = false;
          break;
        }
      }
    }
  } else if (warp < 24) {
    // ---- epilogue ----
    // four warps per accumulator
    const int m = (warp - 16) >> 2, e = (threadIdx.x - 512) & 127;  // e: lane of the accumulator
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const int64_t nhb = 2 * p.nvt;
    grid_dependency_wait();
    for (int64_t i = 0; sm_item(p, i, it); ++i) {
      asm volatile("bar.sync 3, 256;\n" ::: "memory");  // the previous item's rows have been read
      {
        const int k = threadIdx.x - 512;
        const int64_t v = 256 * it.vt + k;
        rows_s[k] = v < 128 * p.nvt ? make_float2(p.sp[v], p.out.row[v].x) : make_float2(0.f, 0.f);
      }
      // one outcome for all eight warps: they share barriers
      if (!tc::bar_and(3, 256, mbar_wait_long(&acc_full[m], (uint32_t)i & 1u, p.err))) break;
      tc::fence_after_sync();
      const int64_t tt = 2 * it.tp + m, n = tt * 128 + e;
      const bool mine = m < it.m && n < p.n;
      const float a = mine ? __ldg(p.tsc + n) * 1.44269504f : 0.f, b = mine ? __ldg(p.out.tok + n) : 0.f;
      // 64 rows of the vocabulary are one 128-byte row of the image
      char* dst = p.out.img + ((tt * nhb + 4 * it.vt) * 128 + e) * 128;
#pragma unroll 1
      for (int c0 = 0; c0 < 256; c0 += 16) {
        uint32_t y[16];
        tc::tmem_ld16_nowait(tbase + 256 * m + lane_off + c0, y);
        tc::tmem_wait_ld(y);
        if (c0 == 240) {
          tc::fence_before_sync();
          tc::mbar_arrive(&acc_empty[m]);
        }
        if (4 * it.vt + (c0 >> 6) >= nhb || m >= it.m) continue;  // (warp-uniform)
#pragma unroll
        for (int k8 = 0; k8 < 2; ++k8) {  // eight rows: one chunk
          uint32_t o[4];
#pragma unroll
          for (int k2 = 0; k2 < 4; ++k2) {
            const int c = 8 * k8 + 2 * k2;
            const float4 f = *reinterpret_cast<const float4*>(rows_s + c0 + c);  // S', log2 |S'| of two
            const float x0 = exp2_approx(fmaf(__uint_as_float(y[c]) * f.x, a, b + f.y));
            const float x1 = exp2_approx(fmaf(__uint_as_float(y[c + 1]) * f.z, a, b + f.w));
            const uint32_t sign = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.z), 0x7030) & 0x80008000u;
            o[k2] = h2_bits(__floats2half2_rn(x0, x1)) ^ sign;
          }
          const int chunk = ((c0 & 63) >> 3) + k8;
          if (mine)
            *reinterpret_cast<uint4*>(dst + (c0 >> 6) * kHStage + (((chunk ^ e) & 7) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  } else if (warp == 24) {
    // ---- H image producer (one thread): each accumulator has its half of the ring ----
    if (lane == 0) {
      grid_dependency_wait();
      constexpr int R = kSH / 2;
      const int64_t tile_bytes = (int64_t)nkbt * 2 * kHStage;
      int64_t nh[2] = {0, 0};
      bool ok = true;
      for (int64_t i = 0; ok && sm_item(p, i, it); ++i) {
        const char* src = p.himg + 2 * it.tp * tile_bytes;
        for (int k = 0; ok && k < 2 * nkbt; ++k, src += kHStage) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (m >= it.m) break;
            const int is = 2 * (int)(nh[m] % R) + m;
            if (nh[m] >= R && !tc::mbar_wait(&h_empty[is], (uint32_t)(nh[m] / R - 1) & 1u, p.err)) {
              ok = false;
              break;
            }
            tc::mbar_arrive_expect_tx(&h_full[is], kHStage);
            tc::bulk_g2s(Hs + is * kHStage, src + m * tile_bytes, kHStage, &h_full[is]);
            ++nh[m];
          }
        }
      }
      if (!ok)
        for (int m = 0; m < 2; ++m)
          for (int64_t q = nh[m] < R ? 0 : nh[m] - R; q < nh[m]; ++q)
            tc::mbar_wait(&h_full[2 * (q % R) + m], (uint32_t)(q / R) & 1u, p.err);
    }
  } else {
    // ---- MMA issuers ----
    const int iw = warp - 25;
    const uint64_t bdesc0 = tc::smem_desc_kmajor_sw128(tc::smem_u32(Ws));
    const uint64_t adesc0 = tc::smem_desc_kmajor_sw128(tc::smem_u32(Hs));
    const uint32_t idesc = tc::idesc_f16_m128(256), d = tbase + 256 * iw;
    int sw = 0, j0 = 0;
    uint32_t pw = 0, ph = 0;
    bool ok = true;
    for (int64_t i = 0; ok && sm_item(p, i, it); ++i) {
      if (i > 0 && !__all_sync(0xffffffffu, tc::mbar_wait(&acc_empty[iw], (uint32_t)(i - 1) & 1u, p.err))) break;
      tc::fence_after_sync();
      const bool active = iw < it.m;  // the second issuer of a lone token tile keeps pace
      for (int k = 0; k < 2 * nkbt; ++k) {
        const int is = 2 * j0 + iw;
        const bool r0 = tc::mbar_try_wait(&w_full[sw], pw), r1 = !active || tc::mbar_try_wait(&h_full[is], ph);
        if (!__all_sync(0xffffffffu, r0 && r1) &&
            !__all_sync(0xffffffffu, tc::mbar_wait(&w_full[sw], pw, p.err) &&
                                         (!active || tc::mbar_wait(&h_full[is], ph, p.err)))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint64_t bd = bdesc0 + (uint64_t)((sw * kStage) >> 4), ad = adesc0 + (uint64_t)((is * kHStage) >> 4);
        if (tc::elect_one()) {
          if (active) {
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_f16_ss(d, ad + ((j * 32) >> 4), bd + ((j * 32) >> 4), idesc, (k | j) != 0);
            tc::mma_commit(&w_empty[sw]);
            tc::mma_commit(&h_empty[is]);
          } else {
            tc::mbar_arrive(&w_empty[sw]);
          }
        }
        __syncwarp();
        if (++sw == kSW) {
          sw = 0;
          pw ^= 1u;
        }
        if (active && ++j0 == kSH / 2) {
          j0 = 0;
          ph ^= 1u;
        }
      }
      if (ok && tc::elect_one()) {
        if (active) tc::mma_commit(&acc_full[iw]);
        else tc::mbar_arrive(&acc_full[iw]);
      }
      __syncwarp();
    }
    if (tc::elect_one()) {
      tc::mma_commit(&mma_done[iw]);
      tc::mbar_wait(&mma_done[iw], 0, p.err);  // every MMA issued here has retired
    }
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 25) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, 512);
  }
}

}  // namespace

cudaError_t launch_softmax_tc(const __half* himg, const float* tsc, const archead_head* head, const Shapes& s,
                              const TcImage& image, unsigned* err, cudaStream_t st, int* launches) {
  if (image.nt != 128) return cudaErrorInvalidValue;
  SoftmaxParams p;
  p.h = *head;
  p.himg = reinterpret_cast<const char*>(himg);
  p.tsc = tsc;
  p.sp = image.sp;
  p.cs = image.cs;
  p.out = image;
  p.n = s.N;
  p.nvt = (s.V + 127) / 128;
  p.ntile = (int)((s.N + 127) / 128);
  p.npair = (p.ntile + 1) / 2;
  p.nkb = (int)(s.D / 128);
  p.nrb = (s.r_c + s.r_r + 31) / 32;
  int gs = 0;
  while ((1 << gs) < s.g) ++gs;
  p.g_shift = gs;
  p.a_words = s.r_c % 4 == 0 && s.r_r % 4 == 0;
  p.err = err;
  int64_t band = (48ll << 20) / (2ll * 2 * kHStage * (p.nkb + p.nrb));  // 48 MB of H, well inside L2
  p.band = (int)(band < 1 ? 1 : (band > p.npair ? p.npair : band));
  p.items = (p.nvt + 1) / 2 * p.npair;
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return e;
  auto kern = s.g == 32 ? softmax_tc_kernel<4> : (s.g == 64 ? softmax_tc_kernel<2> : softmax_tc_kernel<1>);
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmSmem)) != cudaSuccess) return e;
  ++*launches;
  return launch_dependent(kern, p.items < sms ? p.items : sms, kSmThreads, kSmSmem, st, p);
}

}  // namespace archead
