// Gradient product through the packed head on the 5th-generation tensor cores:
//
//   dH[n, d] = s_n ( sum_v dY[n, v] S_v c[v, d / g] q[v, d]  +  sum_j u[n, j] b[j, d] ),
//   u[n, j]  = sum_v dY[n, v] a[v, j],
//
// a = [Q8(A_c) | Q8(A_w)], b = [Q8(B_c) ; Q8(B_w)].  The long axis is the vocabulary, so the
// packed head is a transposed operand: D[n, d] = sum_v A[n, v] B[v, d] with A the FP16 image of
// dY'[n, v] = dY[n, v] S'_v 2^e_n (grad_common.cuh; 128 tokens are the lanes of an accumulator)
// and B the dequantised head, whose vocabulary rows are K and whose columns lie side by side
// (MN-major).  The other way round, with the head as A, few tokens take twice the instructions
// (128 columns each against 256): N = 1 took 190 us against 165 us when both were built on this kernel.
// u is one more tile of columns, whose B, a / S', is prepared once per call in the layout of a W
// stage and copied (built from the INT8 rows in the product's loop it took three times as long as
// a residual tile and set the pace of every round: N = 777, ranks 64 + 64: 3150 us against 760 us).
//
//  * grad_rows_kernel: S'_v per row and their maximum, the factor image.
//  * dy_amax_kernel, dy_image_kernel: the image, from dY or from logits (softmax gradient).
//  * grad_tc_kernel: the product.  A work item is 256 columns x up to 256 tokens (two
//    accumulators) x a slab of the vocabulary; its FP32 sums go to scratch.  (Up to 8 tokens of an
//    SC4 head: grad_warp.cu.)
//  * grad_finish_kernel: adds the slabs in order, adds u b, scales and rounds to BF16.
// Nothing is accumulated in memory, so equal calls give equal bits.
#include "grad_common.cuh"

#include <algorithm>

namespace archead {
namespace {

constexpr int kDequantWarps = 16;
constexpr int kGradThreads = 32 * (kDequantWarps + 7);  // + 4 epilogue, 1 producer, 2 MMA
constexpr int kUnit = 128;                              // vocabulary rows per unit of K
constexpr int kWStage = 32 * 256 * 2;                   // 32 rows x 256 columns FP16
constexpr int kRowBlocks = 592, kRowThreads = 512;      // of grad_rows_kernel

// ---- the image ---------------------------------------------------------------------------
struct RowsParams {
  archead_head h;
  int64_t vpad;
  float* sp;         // S'_v, vpad (0 past V)
  uint32_t* cs;      // 2^(8 - k) per row (grad_row, code_half2) as FP16x2, vpad (0 past V)
  float2* row;       // TcImage's rows without -es, or nullptr
  float* spmax;      // kRowBlocks
  char* fimg;        // factor image, or nullptr without ranks
  int fcols;         // its columns: r_c + r_r rounded up to 64
  int a_words;       // factor rows readable as aligned 32-bit words
};

// Four factor entries j .. j+3 of row v in [A_c | A_w], zeros past r_c + r_r.
__device__ __forceinline__ uint32_t grad_factor_word(const archead_head& h, int a_words, int64_t v, int j) {
  const int rc = h.r_c, rr = h.r_r;
  if (a_words) {
    if (j < rc) return __ldg(reinterpret_cast<const uint32_t*>(h.Ac + v * rc + j));
    if (j < rc + rr) return __ldg(reinterpret_cast<const uint32_t*>(h.Aw + v * rr + (j - rc)));
    return 0u;
  }
  uint32_t w = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int jj = j + u;
    int8_t b = 0;
    if (jj < rc) b = __ldg(h.Ac + v * rc + jj);
    else if (jj < rc + rr) b = __ldg(h.Aw + v * rr + (jj - rc));
    w |= (uint32_t)(uint8_t)b << (8 * u);
  }
  return w;
}

__device__ __forceinline__ GradRow head_row(const archead_head& h, int64_t v, float* sac, float* saw) {
  *sac = h.r_c ? __ldg(h.sAc + v) : 0.f;
  *saw = h.r_r ? __ldg(h.sAw + v) : 0.f;
  return grad_row(bf16_bits_to_float(__ldg(h.r_super + v)), *sac, *saw);
}

__global__ void __launch_bounds__(kRowThreads, 4) grad_rows_kernel(const RowsParams p) {
  allow_dependent_launch();
  __shared__ float red[kRowThreads / 32];
  const int64_t t0 = blockIdx.x * (int64_t)kRowThreads + threadIdx.x, step = gridDim.x * (int64_t)kRowThreads;
  float m = 0.f;
  for (int64_t v = t0; v < p.vpad; v += step) {
    float s = 0.f, c = 0.f;
    if (v < p.h.V) {
      float sac, saw;
      if (p.h.format == ARCHEAD_FMT_ROW8) {
        s = p.h.row_scale[v];
      } else {
        const GradRow gr = head_row(p.h, v, &sac, &saw);
        s = gr.sp;
        c = gr.cs;
      }
    }
    p.sp[v] = s;
    p.cs[v] = h2_bits(__float2half2_rn(256.f * c));
    if (p.row) p.row[v] = make_float2(log2f(fabsf(s)), __uint_as_float(s < 0.f ? 0x80008000u : 0u));
    m = fmaxf(m, fabsf(s));
  }
  if (p.fimg) {  // eight factor entries of a row at a time
    const unsigned per = (unsigned)p.fcols >> 3, total = (unsigned)p.vpad * per;  // < 2^31
#pragma unroll 2
    for (unsigned i = (unsigned)t0; i < total; i += (unsigned)step) {
      const unsigned vi = i / per;
      const int64_t v = vi;
      const int c = (int)(i - vi * per), k = (int)(vi & 31);
      uint32_t o[4] = {0u, 0u, 0u, 0u};
      if (v < p.h.V) {
        float sac, saw;
        const GradRow gr = head_row(p.h, v, &sac, &saw);
        const float rcp = gr.sp != 0.f ? 1.f / gr.sp : 0.f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int j = 8 * c + 4 * q;
          const uint32_t fw = grad_factor_word(p.h, p.a_words, v, j);
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = __fmul_rn((float)(int8_t)((fw >> (8 * e)) & 0xFFu), j + e < p.h.r_c ? sac : saw) * rcp;
          o[2 * q] = h2_bits(__floats2half2_rn(x[0], x[1]));
          o[2 * q + 1] = h2_bits(__floats2half2_rn(x[2], x[3]));
        }
      }
      *reinterpret_cast<uint4*>(p.fimg + (v >> 5) * p.fcols * 64 + (c >> 3) * 4096 + (k >> 3) * 1024 +
                                (k & 7) * 128 + (((c ^ k) & 7) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kRowThreads / 32; ++i) m = fmaxf(m, red[i]);
    p.spmax[blockIdx.x] = m;
  }
  // Nothing here depends on the kernel before, so it runs beside it; the end of this grid has to
  // mean the end of that one for the kernels after.
  grid_dependency_wait();
}

// Exponent of the largest S' (0 for a head of zeros), by one warp.
__device__ __forceinline__ int spmax_exp(const float* spmax) {
  float m = 0.f;
#pragma unroll  // (all loads at once)
  for (int i = 0; i < (kRowBlocks + 31) / 32; ++i) {
    const int b = 32 * i + (threadIdx.x & 31);
    m = fmaxf(m, b < kRowBlocks ? spmax[b] : 0.f);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int e = m > 0.f && m <= 3.402823466e38f ? ilogbf(m) : 0;
  return e < -100 ? -100 : (e > 100 ? 100 : e);  // so that pow2_pair can take every sum of two
}

// Per token the largest |dY| (as bits: a NaN is the largest), one warp per 2048 entries, half of them
// in flight at a time (N = 331, V = 32003: 11 us, cold; with four loads of a lane in flight 13.6).
struct AmaxParams {
  const float* dY;
  int64_t n, V;
  unsigned* amax;
};
template <bool kQuads>
__global__ void __launch_bounds__(256) dy_amax_kernel(const AmaxParams p) {
  const int64_t V = p.V;
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int64_t per = (V + 2047) / 2048, total = per * p.n;
  for (int64_t i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < total; i += gridDim.x * 8ll) {
    const int64_t t = i / per, v0 = (i - t * per) * 2048;
    const float* src = p.dY + t * V + v0;
    const int left = (int)(V - v0 < 2048 ? V - v0 : 2048);
    unsigned m = 0;
    auto take = [&](float x) { m = max(m, __float_as_uint(x) & 0x7fffffffu); };
    if (kQuads) {
#pragma unroll 8
      for (int k = 0; k < 16; ++k) {
        const int v = 128 * k + 4 * lane;
        const float4 x = v < left ? __ldg(reinterpret_cast<const float4*>(src + v)) : make_float4(0.f, 0.f, 0.f, 0.f);
        take(x.x);
        take(x.y);
        take(x.z);
        take(x.w);
      }
    } else {
#pragma unroll 32
      for (int k = 0; k < 64; ++k) {
        const int v = 32 * k + lane;
        take(v < left ? __ldg(src + v) : 0.f);
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) atomicMax(p.amax + t, m);
  }
}

struct ImageParams {
  const float* src;  // dY, or logits
  int64_t n, npad, V;
  int nt, group;
  const float* sp;
  const float* spmax;
  const unsigned* amax;  // dY: per-token maxima
  SoftmaxTokens t;       // logits: dY = exp(Y - lse) - [v = target]
  char* img;
  int* texp;  // per token: dH = 2^texp times the product
  unsigned* err;
};

// Token factor 2^f of the image (before S' 2^-es): dY 2^f S' 2^-es stays below 2^15.
__device__ __forceinline__ int dy_exp(unsigned amax) {
  const int e = (int)(amax >> 23) - 127;  // floor(log2 amax) (subnormal: -127)
  return amax == 0u || amax >= 0x7f800000u ? 0 : 12 - e;
}
// The softmax gradient's entries are below b = 1 - p_target.  p_target comes from the NLL; as
// its FP32 error (a few half steps of the log-sum-exp) may be all of it, b is taken larger.
__device__ __forceinline__ int softmax_exp(float nll, float lse) {
  const float b = fmaxf(fmaxf(-expm1f(-nll), 0x1p-18f), fabsf(lse) * 0x1p-21f);
  return b <= 3.402823466e38f ? 12 - ilogbf(b) : 0;
}

// What the tcgen05 logits kernel needs of the tokens to write the image itself (TcImage), and
// texp.
struct TokensParams {
  int64_t n, V, vpad;
  const float* sp;
  const float* spmax;
  SoftmaxTokens t;
  float* tok;
  int* texp;
  char* img;
  int nt;
  unsigned* err;
};
__global__ void __launch_bounds__(256) grad_tokens_kernel(const TokensParams p) {
  allow_dependent_launch();
  grid_dependency_wait();
  const int es = spmax_exp(p.spmax);
  const int64_t n = blockIdx.x * 256ll + threadIdx.x;
  if (n >= p.n) return;
  const float lse = p.t.lse[n];
  const int32_t t = p.t.targets[n];
  const bool bad = (t < 0 || t >= p.V) && p.t.dnll[n] != 0.f;
  if (bad) atomicOr(p.err, kErrTarget);
  const int f = softmax_exp(p.t.nll[n], lse);
  p.tok[n] = bad ? __int_as_float(0x7fc00000) : fmaf(lse, -1.44269504f, (float)(f - es));
  p.texp[n] = es - f;
}

// The targets' entries: (exp(-nll) - 1) 2^f S'_t 2^-es.
__global__ void __launch_bounds__(256) grad_targets_kernel(const TokensParams p) {
  allow_dependent_launch();
  grid_dependency_wait();
  const int64_t n = blockIdx.x * 256ll + threadIdx.x;
  if (n >= p.n) return;
  const int32_t t = p.t.targets[n];
  if (t < 0 || t >= p.V) return;
  float a, b;
  pow2_pair(-p.texp[n], &a, &b);
  const int64_t tt = n / p.nt;
  *reinterpret_cast<__half*>(p.img + grad_image_offset(tt, t >> 6, p.vpad >> 6, p.nt, (int)(n - tt * p.nt), t & 63)) =
      __float2half_rn(expm1f(-p.t.nll[n]) * a * p.sp[t] * b);
}

// One warp per 128 vocabulary rows and group of 8 tokens, or of 4 where such warps are fewer than run
// at once (a group lies in one image tile): each lane four rows, two 128-byte image rows per token, four
// tokens' loads in flight.  Whole calls with groups of 4 and of 8: nll_grad of 16 tokens, V = 4096, D = 512 32.2 and
// 34.1 us; logits_grad V = 32000, D = 2048 N = 128 (4000 warps of 8) 49.7 and 51.4, N = 600 (20000) 145 and 141; V =
// 128256, D = 4096 N = 128 177 and 171.  Groups of 32 (N = 600 149 us) win nowhere.
template <bool kSoftmax, bool kQuads>
__global__ void __launch_bounds__(256) dy_image_kernel(const ImageParams p) {
  allow_dependent_launch();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t nunits = (p.V + kUnit - 1) / kUnit;
  const int64_t u = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const int64_t n0 = (int64_t)blockIdx.y * p.group;
  const int es = spmax_exp(p.spmax);
  // this lane's token of the group: its factor 2^f and, for logits, lse, target and its entry
  const int64_t mine = n0 + lane;
  int f = 0;
  float lse = 0.f, at = 0.f;
  int32_t target = -1;
  if (lane < p.group && mine < p.n) {
    if (kSoftmax) {
      target = p.t.targets[mine];
      lse = p.t.lse[mine];
      const float nll = p.t.nll[mine];
      f = softmax_exp(nll, lse);
      at = expm1f(-nll);
      if ((target < 0 || target >= p.V) && p.t.dnll[mine] != 0.f) {
        lse = __int_as_float(0x7fc00000);
        if (u == 0) atomicOr(p.err, kErrTarget);
      }
    } else {
      f = dy_exp(p.amax[mine]);
    }
    if (u == 0) p.texp[mine] = es - f;  // within +-240
  }
  if (u >= nunits) return;
  const int64_t v = kUnit * u + 4 * lane;
  const float4 sp = *reinterpret_cast<const float4*>(p.sp + v);
  float e0, e1;
  pow2_pair(-es, &e0, &e1);
  const float s[4] = {sp.x * e0 * e1, sp.y * e0 * e1, sp.z * e0 * e1, sp.w * e0 * e1};
  const int64_t tt = n0 / p.nt;
  const int nn0 = (int)(n0 - tt * p.nt), r = 4 * (lane & 15);  // row in its half unit
  char* dst = p.img + ((tt * 2 * nunits + 2 * u + (lane >> 4)) * p.nt + nn0) * 128 + 2 * (r & 7);
  const float* src = p.src + n0 * p.V + v;
  for (int k0 = 0; k0 < p.group && n0 + k0 < p.npad; k0 += 4) {
    float y[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = n0 + k0 + k < p.n;
      const float* q = src + (k0 + k) * p.V;
      if (kQuads) {
        const float4 x = in && v < p.V ? __ldcs(reinterpret_cast<const float4*>(q)) : make_float4(0.f, 0.f, 0.f, 0.f);
        y[k][0] = x.x;
        y[k][1] = x.y;
        y[k][2] = x.z;
        y[k][3] = x.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[k][e] = in && v + e < p.V ? __ldcs(q + e) : 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t n = n0 + k0 + k;
      const int fk = __shfl_sync(0xffffffffu, f, k0 + k);
      float a, b;
      pow2_pair(fk, &a, &b);
      if (kSoftmax) {
        const float l = __shfl_sync(0xffffffffu, lse, k0 + k), z = __shfl_sync(0xffffffffu, at, k0 + k);
        const int64_t t = __shfl_sync(0xffffffffu, target, k0 + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[k][e] = v + e == t ? z : expf(y[k][e] - l);
          if (v + e >= p.V || n >= p.n) y[k][e] = 0.f;
          if (l != l) y[k][e] = l;
        }
      }
      if (n >= p.npad) break;
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = y[k][e] * a * (b * s[e]);
      const int nn = nn0 + k0 + k;
      *reinterpret_cast<uint2*>(dst + (k0 + k) * 128 + ((((r >> 3) ^ nn) & 7) << 4)) =
          make_uint2(h2_bits(__floats2half2_rn(x[0], x[1])), h2_bits(__floats2half2_rn(x[2], x[3])));
    }
  }
}

// ---- the product -------------------------------------------------------------------------
struct GradParams {
  archead_head h;
  const char* img;
  const uint32_t* cs;
  float* part;  // [slab][n][dp]
  int64_t n, dp;
  int64_t nunits;  // units of 128 vocabulary rows
  int nimg;        // token tiles of the image
  int ntt;         // token tiles of the product: MT tiles of the image each
  int ntiles;      // column tiles: ceil(D / 256), one more for the ranks
  int slabs;
  int g_shift;
  const char* fimg;  // factor image: per 32 rows, fcols x 64 bytes
  int fcols;
  unsigned* err;
};

// IT: tokens per tile of the image (at most 128); MT: image tiles (accumulators) per item.
template <int IT, int MT>
struct GradCfg {
  // Shared memory (227 KB): rings of W stages (32 rows x 256 columns, 16 KB) and image stages (64
  // rows x IT tokens, one per accumulator).  A copy takes about 3000 cycles from the release of its
  // slot (a commit's 700 among them), so the image ring covers five steps of 1024 cycles with two
  // accumulators; the W ring is a multiple of the unit's four stages, so a warp always fills the
  // same slots.  (The packed head goes straight into the warps' registers, a unit ahead: 32 lanes
  // read 512 adjacent bytes.  Through a ring of its own in shared memory, four units deep, the
  // copies' latency set the pace of small batches.)  Two threads issue MMAs, each into its own
  // accumulator of 256 columns: one alone left the tensor cores idle for about 350 cycles between
  // steps (barrier round trips; an issue returns when the MMA before it is nearly done).  With MT =
  // 2 an accumulator is an image tile; with MT = 1 the steps alternate between the two, which the
  // epilogue adds.
  static constexpr int SW = MT == 2 ? 4 : 8;
  static constexpr int SI = MT == 2 ? 10 : (IT == 128 ? 6 : 8);
  static constexpr int ISTAGE = IT * 128;
  static constexpr size_t SMEM = (size_t)SW * kWStage + SI * ISTAGE + 1024 + 512;
  static_assert(SMEM <= 227 * 1024, "does not fit an SM");
  // the MMA reads 128 rows from an image stage: past a smaller one lies the W ring (those lanes
  // are never stored)
  static_assert(SW * kWStage >= 128 * 128, "reads past the last image stage stay inside");
};

struct GradItem {
  int64_t u0, u1;
  int slab, tt, dt;
  int m;      // accumulators
  int cols;   // columns: 256, 128 (the last tile of an odd D / 128) or the ranks' image's
  bool rank;  // the tile of the rank sums
};

template <int MT>
__device__ __forceinline__ bool grad_item(const GradParams& p, int64_t k, GradItem& it) {
  const int64_t i = blockIdx.x + k * gridDim.x;
  const int64_t per = (int64_t)p.ntt * p.ntiles;
  if (i >= per * p.slabs) return false;
  it.slab = (int)(i / per);
  const int64_t r = i - it.slab * per;
  it.tt = (int)(r / p.ntiles);
  it.dt = (int)(r - (int64_t)it.tt * p.ntiles);
  it.u0 = p.nunits * it.slab / p.slabs;
  it.u1 = p.nunits * (it.slab + 1) / p.slabs;
  it.m = p.nimg - it.tt * MT < MT ? p.nimg - it.tt * MT : MT;
  it.rank = it.dt >= (int)((p.h.D + 255) >> 8);
  it.cols = it.rank ? p.fcols : (p.h.D - 256ll * it.dt >= 256 ? 256 : 128);
  return true;
}

// Shared-memory matrix descriptor, MN-major with the 128-byte swizzle: atoms of 64 columns x 8
// rows of K, each K row 128 bytes; lead = byte distance of atoms adjacent in M / N, stride =
// that of atoms adjacent in K.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t lead, uint32_t stride) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lead >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((stride >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

template <int IT, int MT, int CPC>
__global__ void __launch_bounds__(kGradThreads, 1) grad_tc_kernel(const GradParams p) {
  using C = GradCfg<IT, MT>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* Is = smem;
  unsigned char* Ws = Is + C::SI * C::ISTAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(Ws + C::SW * kWStage);
  uint64_t* w_full = bars;
  uint64_t* w_empty = w_full + C::SW;
  uint64_t* i_full = w_empty + C::SW;
  uint64_t* i_empty = i_full + C::SI;
  uint64_t* acc_full = i_empty + C::SI;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* mma_done = acc_empty + 1;  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::SW; ++i) {
      tc::mbar_init(&w_full[i], MT == 2 ? 4 : 2);  // the warps that fill a stage
      tc::mbar_init(&w_empty[i], MT);              // the issuers that read it
    }
    for (int i = 0; i < C::SI; ++i) {
      tc::mbar_init(&i_full[i], 1);
      tc::mbar_init(&i_empty[i], 1);
    }
    tc::mbar_init(acc_full, 2);
    tc::mbar_init(acc_empty, 128);
    tc::mbar_init(&mma_done[0], 1);
    tc::mbar_init(&mma_done[1], 1);
    tc::mbar_fence_init();
  }
  if (warp == kDequantWarps + 5) tc::tmem_alloc(tmem_slot, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  GradItem it;

  if (warp < kDequantWarps) {
    // ---- dequantisation: lane = vocabulary row of a 32-row group ----
    // A warp owns rows 32 rg .. + 31 (a W stage) and one 128-column block b: with two accumulators
    // half of that block's 16-byte chunks in every unit; with one, where units follow one another
    // twice as fast, all of them in every other unit, which halves what a unit pays for barriers
    // and fences (one token: 148 -> 141 us).
    constexpr int NH = 3 - MT;  // halves of the chunks per warp, and groups of warps by unit
    const int rg = warp & 3, b = (warp >> 2) & 1, grp = warp >> 3;
    const int s = 32 * rg + lane;  // row in the unit
    const int slot = NH == 2 ? 4 * grp + rg : rg;  // its place in the W ring (one or two units)
    static_assert(C::SW == 4 * NH, "a slot belongs to one group of warps");
    // The lane's 128-byte row of the slot, with its swizzle: chunk j of the block's first 64-column
    // atom is stored at w_addr ^ 16 j, of the second 4096 bytes on.
    const uint32_t w_addr = tc::smem_u32(Ws) + (uint32_t)(slot * kWStage + b * 2 * 4096 + (lane >> 3) * 1024 +
                                                          (lane & 7) * 128 + ((lane & 7) << 4));
    uint32_t wp = 1;  // parity of the slot's last release (the first use waits for none)
    int64_t seq = 0;  // units of this CTA so far
    bool copied = false;  // a copy from the factor image was the slot's last use
    bool ok = true;
    grid_dependency_wait();  // the row table and the factor image come from kernels before this
    for (int64_t i = 0; ok && grad_item<MT>(p, i, it); ++i) {
      // this warp's units of the item
      const int64_t ua = NH == 2 ? it.u0 + ((seq ^ grp) & 1) : it.u0;
      seq += it.u1 - it.u0;
      if (it.rank) {
        // Whole stages from the factor image, copied by one of a stage's warps; the others only
        // keep pace (a warp that skipped stages would lose count of the phases).
        const uint32_t bytes = (uint32_t)p.fcols * 64u;
        for (int64_t u = ua; u < it.u1; u += NH) {
          if (!__all_sync(0xffffffffu, tc::mbar_wait(&w_empty[slot], wp, p.err))) {
            ok = false;
            break;
          }
          if (lane == 0) {
            if (b == 0 && (NH == 2 || grp == 0)) {
              tc::mbar_arrive_expect_tx(&w_full[slot], bytes);
              tc::bulk_g2s(Ws + slot * kWStage, p.fimg + (4 * u + rg) * bytes, bytes, &w_full[slot]);
              copied = true;
            } else {
              tc::mbar_arrive(&w_full[slot]);
            }
          }
          __syncwarp();
          wp ^= 1u;
        }
        continue;
      }
      const bool work = 128 * b < it.cols;
      const int64_t col = 256ll * it.dt + (work ? 128 * b : 0);
      // One unit ahead: the next unit's packed chunks, codes and scale are on their way while this
      // unit's entries are made, each loaded where the one before has been used up.
      // (rows past V are padded, in cs as in the codes)
      const int64_t G = p.h.D >> p.g_shift;
      const uint32_t* cs_at = p.cs + ua * kUnit + s;
      const uint8_t* code_at = p.h.r_code + (ua * kUnit + s) * G + (col >> p.g_shift);
      uint32_t codes = 0, cs = 0;
      if (CPC != 0 && ua < it.u1) {
        codes = load_codes<CPC>(code_at);
        cs = load_word(cs_at);
      }
      const int64_t tile = (p.h.D >> 7) << 13;  // bytes of a 128-row tile
      const uint8_t* p_at = p.h.r_nib + ua * tile + ((col >> 7) << 13) + s * 16;
      uint4 q[2 * NH];
      if (CPC != 0 && ua < it.u1) {
#pragma unroll
        for (int c = 0; c < 2 * NH; ++c) q[c] = ldg_stream(p_at + (NH == 2 ? c : 2 * grp + c) * 2048);
      }
      for (int64_t u = ua; u < it.u1; u += NH) {
        const int64_t v = u * kUnit + s;
        const bool more = u + NH < it.u1;
        const bool w_ready = tc::mbar_test(&w_empty[slot], wp);
        const uint32_t now = codes, now_cs = cs;
        if (CPC != 0 && more) {
          code_at += NH * kUnit * G;
          cs_at += NH * kUnit;
          p_at += NH * tile;
          codes = load_codes<CPC>(code_at);
          cs = load_word(cs_at);
        }
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
          const int ch = NH == 2 ? hh : grp;  // half of the block's chunks
          // The entries are made in registers before the wait for the stage's slot, so a slot is
          // empty only for the stores.
          uint32_t o[8][4];  // 16-byte chunks of eight columns
          if (CPC != 0) {
            if (work) {
#pragma unroll
              for (int wn = 0; wn < 4; ++wn) {  // window of 32 columns
                const __half2 c2 = code_half2(now, CPC == 1 ? 0 : (CPC == 2 ? wn >> 1 : wn), now_cs);
                const __half2 nc24 = __hmul2(c2, __float2half2_rn(-24.f));
#pragma unroll
                for (int c = 0; c < 2; ++c) {  // columns 32 wn + 16 ch + 8 c .. + 7
                  const uint4 x = q[2 * hh + c];
                  const uint32_t word = wn == 0 ? x.x : (wn == 1 ? x.y : (wn == 2 ? x.z : x.w));
                  __half2 e[4];
                  dequant_word(word, c2, nc24, e);
#pragma unroll
                  for (int j = 0; j < 4; ++j) o[2 * wn + c][j] = h2_bits(e[j]);
                }
              }
            }
            if (more) {
#pragma unroll
              for (int c = 0; c < 2; ++c)
                q[2 * hh + c] = ldg_stream(p_at + (NH == 2 ? 2 * hh + c : 2 * grp + c) * 2048);
            }
          } else if (work) {  // INT8 rows straight from global memory
            const uint4* src = reinterpret_cast<const uint4*>(p.h.r_nib + v * p.h.D + col) + 4 * ch;
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // 16 columns: chunks 2c, 2c + 1 of the half block
              const uint4 raw = v < p.h.V ? ldg_stream(src + c) : make_uint4(0, 0, 0, 0);
              const uint32_t x[4] = {raw.x ^ 0x80808080u, raw.y ^ 0x80808080u, raw.z ^ 0x80808080u, raw.w ^ 0x80808080u};
#pragma unroll
              for (int j = 0; j < 8; ++j)
                o[2 * c + (j >> 2)][j & 3] = h2_bits(bytes_to_half2(x[j >> 1], (j & 1) ? 0x4342 : 0x4140));
            }
          }
          if (hh == 0 && !__all_sync(0xffffffffu, w_ready) &&
              !__all_sync(0xffffffffu, tc::mbar_wait(&w_empty[slot], wp, p.err)))
            ok = false;
          if (!ok) break;
          if (work) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              // SC4: columns 32 (c / 2) + 16 ch + 8 (c % 2), a chunk of atom c / 4; INT8: chunk c of
              // atom ch
              const int atom = CPC != 0 ? c >> 2 : ch;
              const int chunk = CPC != 0 ? ((c >> 1) & 1) * 4 + 2 * ch + (c & 1) : c;
              st_shared16((w_addr ^ (uint32_t)(chunk << 4)) + atom * 4096, o[c][0], o[c][1], o[c][2], o[c][3]);
            }
          }
        }
        if (!ok) break;
        tc::fence_proxy_async_smem();  // the MMA reads the stage through the async proxy
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&w_full[slot]);
        wp ^= 1u;
        copied = false;
      }
    }
    if (!ok && copied) tc::mbar_wait(&w_full[slot], wp, p.err);  // the copy may be in flight
  } else if (warp < kDequantWarps + 4) {
    // ---- epilogue: lane = token; raw sums to scratch ----
    const int e = warp - kDequantWarps;
    const uint32_t lane_off = (uint32_t)(32 * e) << 16;
    for (int64_t i = 0; grad_item<MT>(p, i, it); ++i) {
      if (!tc::bar_and(1, 128, mbar_wait_long(acc_full, (uint32_t)i & 1u, p.err))) break;
      tc::fence_after_sync();
      const int RR = p.h.r_c + p.h.r_r;
      const int live = it.rank ? (RR + 3) & ~3 : it.cols;  // (rows of scratch end on a multiple of 4)
      const int t = 32 * e + lane;
#pragma unroll 1
      for (int m = 0; m < it.m; ++m) {
        const int64_t n = ((int64_t)it.tt * MT + m) * IT + t;
        const bool mine = t < IT && n < p.n;
        float* dst = p.part + ((int64_t)it.slab * p.n + n) * p.dp + (it.rank ? p.h.D : 256ll * it.dt);
        if (32 * e >= IT) break;  // (warp-uniform)
#pragma unroll 1
        for (int c0 = 0; c0 < it.cols; c0 += 16) {
          float y[16];
          tc::tmem_ld16(tbase + m * 256 + lane_off + c0, y);
          if (MT == 1) {  // the odd steps' sums
            float z[16];
            tc::tmem_ld16(tbase + 256 + lane_off + c0, z);
#pragma unroll
            for (int q = 0; q < 16; ++q) y[q] += z[q];
          }
          if (mine) {
#pragma unroll
            for (int q = 0; q < 16; q += 4)
              if (c0 + q < live)
                __stcs(reinterpret_cast<float4*>(dst + c0 + q), make_float4(y[q], y[q + 1], y[q + 2], y[q + 3]));
          }
        }
      }
      tc::fence_before_sync();
      tc::mbar_arrive(acc_empty);
    }
  } else if (warp == kDequantWarps + 4) {
    // ---- image producer (one thread); the image comes from the kernel before this one ----
    if (lane == 0) {
      grid_dependency_wait();
      const int64_t tile_bytes = p.nunits * 2 * C::ISTAGE;
      // With MT = 2 each accumulator has its own half of the ring (slot 2 j + m), so that an item
      // with one image tile leaves the other's place as it is.
      constexpr int R = C::SI / MT;
      int64_t ni[MT] = {};
      bool ok = true;
      for (int64_t i = 0; ok && grad_item<MT>(p, i, it); ++i) {
        const char* src = p.img + (int64_t)it.tt * MT * tile_bytes + 2 * it.u0 * C::ISTAGE;
        for (int64_t u = 2 * it.u0; ok && u < 2 * it.u1; ++u, src += C::ISTAGE) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if (m >= it.m) break;
            const int is = (int)(ni[m] % R) * MT + m;
            if (ni[m] >= R && !tc::mbar_wait(&i_empty[is], (uint32_t)(ni[m] / R - 1) & 1u, p.err)) {
              ok = false;
              break;
            }
            tc::mbar_arrive_expect_tx(&i_full[is], C::ISTAGE);
            tc::bulk_g2s(Is + is * C::ISTAGE, src + m * tile_bytes, C::ISTAGE, &i_full[is]);
            ++ni[m];
          }
        }
      }
      if (!ok)
        for (int m = 0; m < MT; ++m)
          for (int64_t q = ni[m] < R ? 0 : ni[m] - R; q < ni[m]; ++q)
            tc::mbar_wait(&i_full[(q % R) * MT + m], (uint32_t)(q / R) & 1u, p.err);
    }
  } else {
    // ---- MMA issuers: two warps, one elected lane of each issues ----
    // A step is 64 rows: two W stages and one image stage per accumulator.  Its barriers are
    // probed together, then one thread issues the step.  With MT = 2 issuer iw takes image tile iw
    // in every step, with MT = 1 the steps kk = iw mod 2.
    const int iw = warp - (kDequantWarps + 5);
    const uint64_t bdesc0 = desc_mn_sw128(tc::smem_u32(Ws), 4096, 1024);
    const uint64_t adesc0 = tc::smem_desc_kmajor_sw128(tc::smem_u32(Is));
    constexpr int R = C::SI / 2;  // this issuer's slots of the image ring: 2 j + iw
    const uint32_t d = tbase + 256 * iw;
    int sw = MT == 2 ? 0 : 2 * iw, j0 = 0;
    uint32_t pw = 0, pi = 0;
    bool ok = true;
    for (int64_t i = 0; ok && grad_item<MT>(p, i, it); ++i) {
      if (i > 0 && !__all_sync(0xffffffffu, tc::mbar_wait(acc_empty, (uint32_t)(i - 1) & 1u, p.err))) break;
      tc::fence_after_sync();
      const uint32_t idesc = tc::idesc_f16_m128(it.cols) | (1u << 16);  // B is MN-major
      const bool active = MT == 1 || iw < it.m;  // the second issuer of a lone image tile keeps pace
      const int64_t k1 = 2 * (it.u1 - it.u0);
      for (int64_t kk = MT == 2 ? 0 : iw; kk < k1; kk += 3 - MT) {
        const int is = 2 * j0 + iw;
        const bool r0 = tc::mbar_try_wait(&w_full[sw], pw), r1 = tc::mbar_try_wait(&w_full[sw + 1], pw);
        const bool r2 = !active || tc::mbar_try_wait(&i_full[is], pi);
        if (!__all_sync(0xffffffffu, r0 && r1 && r2) &&
            !__all_sync(0xffffffffu, tc::mbar_wait(&w_full[sw], pw, p.err) && tc::mbar_wait(&w_full[sw + 1], pw, p.err) &&
                                         (!active || tc::mbar_wait(&i_full[is], pi, p.err)))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint64_t bd = bdesc0 + (uint64_t)((sw * kWStage) >> 4);
        const uint64_t ad = adesc0 + (uint64_t)((is * C::ISTAGE) >> 4);
        if (tc::elect_one()) {
          if (active) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // K steps of 16 rows: 32 bytes of A, two 8-row atoms of B
              mma_f16_ss(d, ad + ((j * 32) >> 4), bd + (uint64_t)(((j >> 1) * kWStage + (j & 1) * 2048) >> 4), idesc,
                         kk >= 3 - MT || j != 0);
              if (j == 1) tc::mma_commit(&w_empty[sw]);
            }
            tc::mma_commit(&w_empty[sw + 1]);
            tc::mma_commit(&i_empty[is]);
          } else {
            tc::mbar_arrive(&w_empty[sw]);
            tc::mbar_arrive(&w_empty[sw + 1]);
          }
        }
        __syncwarp();
        sw += MT == 2 ? 2 : 4;
        if (sw >= C::SW) {
          sw -= C::SW;
          pw ^= 1u;
        }
        if (active && ++j0 == R) {
          j0 = 0;
          pi ^= 1u;
        }
      }
      if (ok && tc::elect_one()) {
        if (active) tc::mma_commit(acc_full);
        else tc::mbar_arrive(acc_full);
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
  if (warp == kDequantWarps + 5) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, 512);
  }
}

// ---- finish ------------------------------------------------------------------------------
struct FinishParams {
  archead_head h;
  const float* part;
  int64_t n, dp;
  int slabs;
  const int* texp;
  const float* rowscale;
  __nv_bfloat16* dH;
};

__device__ __forceinline__ void mma_bf16_16816(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf2_bits(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }

// 16 MT tokens x 128 columns per block, a warp per 32 columns (one group of B's scales).  The
// rank product runs as warp MMAs: the INT8 entries of b are exact in BF16, and u times the scale
// is split into two BF16 pieces (16 bits, against the 8 that the result keeps).  Memory bounds it
// (each slab's sums are read once); on the CUDA cores, one column pair and 16 tokens per thread,
// the product took three times as long, and a lone block of a small batch 40 us of dependent
// loads.
constexpr int kFinishPad = 4;  // floats after a row of u
constexpr int kFinishRow = 132;  // floats per token of the columns' sums (MT = 1)
// With 16 tokens per block (few tokens or columns) latency counts, so 512 threads add the slabs, one
// float4 of the columns and one of u each, and hand them to the four warps through shared memory
// (N = 166, D = 512, 133 ranks, 38 slabs: 57 us with 128 threads for either).
constexpr int finish_threads(int mt) { return mt == 1 ? 512 : 128; }
template <int MT>
__global__ void __launch_bounds__(finish_threads(MT)) grad_finish_kernel(const FinishParams p) {
  constexpr int T = finish_threads(MT);
  extern __shared__ __align__(16) unsigned char fsm[];
  const int RR = p.h.r_c + p.h.r_r, rp = (RR + 15) & ~15, us_row = rp + kFinishPad;
  float* us = reinterpret_cast<float*>(fsm);                      // [16 MT][us_row]
  float* ss = us + 16 * MT * us_row;                              // [rp][4] scales of b
  int8_t* bs = reinterpret_cast<int8_t*>(ss + 4 * rp);            // [rp][144] entries of b
  float* ms = reinterpret_cast<float*>(bs + 144 * rp);            // [16][kFinishRow] with MT = 1
  const int64_t n0 = blockIdx.x * (16ll * MT), d0 = blockIdx.y * 128ll;
  const int64_t G = p.h.D / p.h.g;
  for (int i = threadIdx.x; i < rp * 8; i += T) {  // b does not depend on earlier kernels
    const int j = i >> 3, c = i & 7;
    const bool core = j < p.h.r_c;
    uint4 q = make_uint4(0, 0, 0, 0);
    if (j < RR)
      q = __ldg(reinterpret_cast<const uint4*>((core ? p.h.Bc + j * p.h.D : p.h.Bw + (j - p.h.r_c) * p.h.D) + d0) + c);
    *reinterpret_cast<uint4*>(bs + j * 144 + 16 * c) = q;
  }
  for (int i = threadIdx.x; i < rp * 4; i += T) {
    const int j = i >> 2;
    const bool core = j < p.h.r_c;
    const int64_t grp = (d0 + 32 * (i & 3)) / p.h.g;
    ss[i] = j < RR ? __ldg((core ? p.h.sBc + j * G : p.h.sBw + (j - p.h.r_c) * G) + grp) : 0.f;
  }
  grid_dependency_wait();
  const int64_t slab = p.n * p.dp;
  // u: four ranks of a token of the block
  const int uq = rp > 0 ? rp >> 2 : 1;  // quads of a token
  auto u_at = [&](int i, int* t, int* j) {
    *t = i / uq;
    *j = 4 * (i - *t * uq);
    return i < 4 * MT * rp && n0 + *t < p.n && *j < RR ? p.part + (n0 + *t) * p.dp + p.h.D + *j : nullptr;
  };
  auto u_put = [&](int t, int j, float4 a) {
    if (j + 1 >= RR) a.y = 0.f;  // past the ranks nothing was written
    if (j + 2 >= RR) a.z = 0.f;
    if (j + 3 >= RR) a.w = 0.f;
    *reinterpret_cast<float4*>(us + t * us_row + j) = a;
  };
  auto add = [](float4& a, const float* x) {
    const float4 y = __ldcs(reinterpret_cast<const float4*>(x));
    a.x += y.x;
    a.y += y.y;
    a.z += y.z;
    a.w += y.w;
  };
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  int first = threadIdx.x;
  if (MT == 1) {
    const int mt = threadIdx.x >> 5, mc = 4 * (threadIdx.x & 31);
    const float* msrc = n0 + mt < p.n ? p.part + (n0 + mt) * p.dp + d0 + mc : nullptr;
    int t, j;
    const float* usrc = u_at(threadIdx.x, &t, &j);
    float4 m = zero, u = zero;
#pragma unroll 8
    for (int s = 0; s < p.slabs; ++s) {
      if (msrc) add(m, msrc + s * slab);
      if (usrc) add(u, usrc + s * slab);
    }
    *reinterpret_cast<float4*>(ms + mt * kFinishRow + mc) = m;
    if (first < 4 * rp) u_put(t, j, u);
    first += T;
  }
  for (int i = first; i < 4 * MT * rp; i += T) {
    int t, j;
    const float* src = u_at(i, &t, &j);
    float4 a = zero;
    if (src)
#pragma unroll 8
      for (int s = 0; s < p.slabs; ++s) add(a, src + s * slab);
    u_put(t, j, a);
  }
  if (MT == 1) {
    __syncthreads();
    if (threadIdx.x >= 128) return;
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, gr = lane >> 2, q = lane & 3;
  float acc[MT][4][4];
  int ex[MT][2];  // the rows' exponents and scales, needed last
  float sc[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int hrow = 0; hrow < 2; ++hrow) {
      const int64_t n = n0 + 16 * m + 8 * hrow + gr;
      ex[m][hrow] = n < p.n ? p.texp[n] : 0;
      sc[m][hrow] = n < p.n && p.rowscale ? p.rowscale[n] : 1.f;
    }
  if (MT == 1) {
#pragma unroll
    for (int hrow = 0; hrow < 2; ++hrow)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 x = *reinterpret_cast<const float2*>(ms + (8 * hrow + gr) * kFinishRow + 32 * w + 8 * c + 2 * q);
        acc[0][c][2 * hrow] = x.x;
        acc[0][c][2 * hrow + 1] = x.y;
      }
  }
#pragma unroll
  for (int m = 0; MT > 1 && m < MT; ++m) {
    float2 a[2][4];
    const float* src[2];
    bool in[2];
#pragma unroll
    for (int hrow = 0; hrow < 2; ++hrow) {
      const int64_t n = n0 + 16 * m + 8 * hrow + gr;
      in[hrow] = n < p.n;
      src[hrow] = p.part + n * p.dp + d0 + 32 * w + 2 * q;
#pragma unroll
      for (int c = 0; c < 4; ++c) a[hrow][c] = make_float2(0.f, 0.f);
    }
#pragma unroll 2
    for (int s = 0; s < p.slabs; ++s)
#pragma unroll
      for (int hrow = 0; hrow < 2; ++hrow)
        if (in[hrow])
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 x = __ldcs(reinterpret_cast<const float2*>(src[hrow] + s * slab + 8 * c));
            a[hrow][c].x += x.x;
            a[hrow][c].y += x.y;
          }
#pragma unroll
    for (int hrow = 0; hrow < 2; ++hrow)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[m][c][2 * hrow] = a[hrow][c].x;
        acc[m][c][2 * hrow + 1] = a[hrow][c].y;
      }
  }
  if (MT > 1) __syncthreads();
  for (int k0 = 0; k0 < rp; k0 += 16) {
    const int j = k0 + 2 * q;
    uint32_t b[4][2];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int8_t* src = bs + j * 144 + 32 * w + 8 * c + gr;
      b[c][0] = bf2_bits(__floats2bfloat162_rn((float)src[0], (float)src[144]));
      b[c][1] = bf2_bits(__floats2bfloat162_rn((float)src[8 * 144], (float)src[9 * 144]));
    }
    const float s[4] = {ss[4 * j + w], ss[4 * (j + 1) + w], ss[4 * (j + 8) + w], ss[4 * (j + 9) + w]};
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // rows gr, gr + 8; k 2q, 2q + 8
        const float2 u = *reinterpret_cast<const float2*>(us + (16 * m + gr + 8 * (e & 1)) * us_row + j + 8 * (e >> 1));
        const float x = u.x * s[2 * (e >> 1)], y = u.y * s[2 * (e >> 1) + 1];
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        hi[e] = bf2_bits(h);
        lo[e] = bf2_bits(__floats2bfloat162_rn(x - __low2float(h), y - __high2float(h)));
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mma_bf16_16816(acc[m][c], hi, b[c][0], b[c][1]);
        mma_bf16_16816(acc[m][c], lo, b[c][0], b[c][1]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int hrow = 0; hrow < 2; ++hrow) {
      const int64_t n = n0 + 16 * m + 8 * hrow + gr;
      if (n >= p.n) continue;
      const float f = sc[m][hrow];
      float e0, e1;
      pow2_pair(ex[m][hrow], &e0, &e1);
      __nv_bfloat16* dst = p.dH + n * p.h.D + d0 + 32 * w + 2 * q;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float x = acc[m][c][2 * hrow] * e0 * e1 * f, y = acc[m][c][2 * hrow + 1] * e0 * e1 * f;
        *reinterpret_cast<__nv_bfloat162*>(dst + 8 * c) = __floats2bfloat162_rn(f == 0.f ? 0.f : x, f == 0.f ? 0.f : y);
      }
    }
}

size_t finish_smem(int mt, int RR) {
  const size_t rp = (RR + 15) / 16 * 16;
  return 16 * mt * (rp + kFinishPad) * 4 + rp * 16 + rp * 144 + (mt == 1 ? 16 * kFinishRow * 4 : 0);
}

// ---- host --------------------------------------------------------------------------------
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

struct GradPlan {
  bool warp;   // on warp MMAs (grad_warp.cu)
  int it, mt;  // tokens per image tile, image tiles per item
  int nimg, ntt, ntiles, slabs;
  int64_t npad, nunits, dp;
  int fcols;
  size_t o_img, o_fimg, o_sp, o_cs, o_row, o_spmax, o_amax, o_texp, o_tok, o_part, bytes;
};

GradPlan grad_plan(const archead_head& h, int64_t n) {
  GradPlan g;
  const int RR = h.r_c + h.r_r;
  g.it = head_grad_image_tile(n);
  g.mt = n <= 128 ? 1 : 2;
  g.nimg = (int)((n + g.it - 1) / g.it);
  g.ntt = (g.nimg + g.mt - 1) / g.mt;
  g.npad = (int64_t)g.nimg * g.it;
  g.ntiles = (int)((h.D + 255) / 256) + (RR > 0);
  g.nunits = (h.V + kUnit - 1) / kUnit;
  g.dp = (h.D + RR + 3) / 4 * 4;
  // Slabs of the vocabulary: CTAs run items of equal length side by side, so the time is that of
  // ceil(items / CTAs) rounds, each of 1 / slabs of a tile's units and about 6 us for filling the
  // pipeline and storing the sums, plus the sums' way through memory.  Measured: 1.6 us per unit
  // of 128 rows with two accumulators, 0.9 us with one.
  const int64_t tiles = (int64_t)g.ntt * g.ntiles;
  const int64_t sms = sm_count();
  g.slabs = 1;
  // The warp MMAs win up to 8 tokens, a whole call by 143 -> 128 us at N = 1 and 146 -> 134 us at
  // N = 8 (V = 151936, D = 4096); with 16 they need twice the registers: 155 -> 200 us.
  g.warp = n <= 8 && h.format == ARCHEAD_FMT_SC4;
  if (g.warp) {  // one round of CTAs, each at least four units
    const int64_t all = (h.D + 255) / 256 + (RR + 63) / 64;
    g.slabs = (int)std::max<int64_t>(1, std::min(sms * kGradWarpCtas / all, g.nunits / 4));
  }
  double best = 1e300;
  for (int s = 1; !g.warp && s <= 64 && s * 4 <= g.nunits + 3; ++s) {
    if (s > 1 && 4.0 * s * n * g.dp > 1e9) break;  // (scratch)
    const int64_t rounds = (tiles * s + sms - 1) / sms;
    const double tile_us = g.nunits * (g.mt == 2 ? 1.6 : 0.9);
    const double cost = rounds * (tile_us / s + 6.0) + 8.0 * s * n * g.dp / 4e6 + 0.3 * s;
    if (cost < best * 0.995) {
      best = cost;
      g.slabs = s;
    }
  }
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t r = o;
    o += up256(b);
    return r;
  };
  g.o_img = take((size_t)g.npad * g.nunits * kUnit * 2);
  g.fcols = (RR + 63) / 64 * 64;
  g.o_fimg = take((size_t)g.nunits * kUnit * g.fcols * 2);
  g.o_sp = take((size_t)g.nunits * kUnit * 4);
  g.o_cs = take((size_t)g.nunits * kUnit * 4);
  g.o_row = take((size_t)g.nunits * kUnit * 8);
  g.o_spmax = take(kRowBlocks * 4);
  g.o_amax = take((size_t)n * 4);
  g.o_texp = take((size_t)n * 4);
  g.o_tok = take((size_t)n * 4);
  g.o_part = take((size_t)g.slabs * n * g.dp * 4);
  g.bytes = o;
  return g;
}

template <typename Kern, typename Params>
cudaError_t launch_pdl(Kern kern, dim3 grid, int threads, size_t smem, cudaStream_t st, const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int IT, int MT, int CPC>
cudaError_t launch_grad_cfg(const GradParams& p, cudaStream_t st) {
  auto kern = grad_tc_kernel<IT, MT, CPC>;
  constexpr size_t smem = GradCfg<IT, MT>::SMEM;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)p.ntt * p.ntiles * p.slabs, sms = sm_count();
  return launch_pdl(kern, dim3((unsigned)(items < sms ? items : sms)), kGradThreads, smem, st, p);
}

template <int IT, int MT>
cudaError_t launch_grad_it(const GradParams& p, cudaStream_t st) {
  if (p.h.format == ARCHEAD_FMT_ROW8) return launch_grad_cfg<IT, MT, 0>(p, st);
  if (p.h.g == 32) return launch_grad_cfg<IT, MT, 4>(p, st);
  if (p.h.g == 64) return launch_grad_cfg<IT, MT, 2>(p, st);
  return launch_grad_cfg<IT, MT, 1>(p, st);
}

struct GradParts {
  char *img, *fimg;
  float *sp, *spmax, *tok, *part;
  uint32_t* cs;
  float2* row;
  unsigned* amax;
  int* texp;
};
GradParts grad_parts(const HeadGrad& a, const GradPlan& g) {
  char* b = a.scratch;
  GradParts q;
  q.img = b + g.o_img;
  q.fimg = b + g.o_fimg;
  q.sp = reinterpret_cast<float*>(b + g.o_sp);
  q.cs = reinterpret_cast<uint32_t*>(b + g.o_cs);
  q.spmax = reinterpret_cast<float*>(b + g.o_spmax);
  q.tok = reinterpret_cast<float*>(b + g.o_tok);
  q.part = reinterpret_cast<float*>(b + g.o_part);
  q.row = reinterpret_cast<float2*>(b + g.o_row);
  q.amax = reinterpret_cast<unsigned*>(b + g.o_amax);
  q.texp = reinterpret_cast<int*>(b + g.o_texp);
  return q;
}

TokensParams tokens_params(const HeadGrad& a, const SoftmaxTokens& t) {
  const GradPlan g = grad_plan(*a.head, a.n);
  const GradParts b = grad_parts(a, g);
  return {a.n, a.head->V, g.nunits * kUnit, b.sp, b.spmax, t, b.tok, b.texp, b.img, g.it, a.err};
}

// Rows of src readable as 16-byte words.
bool image_quads(const HeadGrad& a, const float* src) {
  return a.head->V % 4 == 0 && reinterpret_cast<uintptr_t>(src) % 16 == 0;
}

cudaError_t grad_image(const HeadGrad& a, const float* src, const SoftmaxTokens* t) {
  const GradPlan g = grad_plan(*a.head, a.n);
  const GradParts b = grad_parts(a, g);
  const int group = g.nunits * (g.npad / 8) < 40ll * sm_count() ? 4 : 8;
  const ImageParams p = {src, a.n, g.npad, a.head->V, g.it, group, b.sp, b.spmax, b.amax,
                         t ? *t : SoftmaxTokens{}, b.img, b.texp, a.err};
  const dim3 grid((unsigned)((g.nunits + 7) / 8), (unsigned)(g.npad / group));
  const bool quads = image_quads(a, src);
  ++*a.launches;
  if (t)
    return quads ? launch_pdl(dy_image_kernel<true, true>, grid, 256, 0, a.st, p)
                 : launch_pdl(dy_image_kernel<true, false>, grid, 256, 0, a.st, p);
  return quads ? launch_pdl(dy_image_kernel<false, true>, grid, 256, 0, a.st, p)
               : launch_pdl(dy_image_kernel<false, false>, grid, 256, 0, a.st, p);
}

}  // namespace

int head_grad_image_tile(int64_t n) { return n <= 16 ? 16 : (n <= 32 ? 32 : (n <= 64 ? 64 : 128)); }

size_t head_grad_scratch_bytes(const archead_head* head, int64_t n) { return grad_plan(*head, n).bytes; }

cudaError_t grad_rows(const HeadGrad& a) {
  const archead_head& h = *a.head;
  const GradPlan g = grad_plan(h, a.n);
  const GradParts b = grad_parts(a, g);
  const RowsParams p = {h, g.nunits * kUnit, b.sp, b.cs, b.row, b.spmax,
                        g.fcols ? b.fimg : nullptr, g.fcols, h.r_c % 4 == 0 && h.r_r % 4 == 0};
  ++*a.launches;
  return launch_pdl(grad_rows_kernel, dim3(kRowBlocks), kRowThreads, 0, a.st, p);
}

cudaError_t grad_amax(const HeadGrad& a, const float* dY) {
  const GradParts b = grad_parts(a, grad_plan(*a.head, a.n));
  cudaError_t e = cudaMemsetAsync(b.amax, 0, (size_t)a.n * 4, a.st);
  if (e != cudaSuccess) return e;
  const int64_t blocks = ((a.head->V + 2047) / 2048 * a.n + 7) / 8;
  const AmaxParams p = {dY, a.n, a.head->V, b.amax};
  auto kern = image_quads(a, dY) ? dy_amax_kernel<true> : dy_amax_kernel<false>;
  kern<<<(unsigned)(blocks < 148 * 16 ? blocks : 148 * 16), 256, 0, a.st>>>(p);
  ++*a.launches;
  return cudaGetLastError();
}

cudaError_t grad_image_dy(const HeadGrad& a, const float* dY) { return grad_image(a, dY, nullptr); }

cudaError_t grad_image_softmax(const HeadGrad& a, const float* logits, const SoftmaxTokens& t) {
  return grad_image(a, logits, &t);
}

cudaError_t grad_tokens(const HeadGrad& a, const SoftmaxTokens& t, TcImage* image) {
  const TokensParams p = tokens_params(a, t);
  const GradParts b = grad_parts(a, grad_plan(*a.head, a.n));
  *image = TcImage{p.img, b.row, p.tok, p.nt, p.sp, b.cs};
  ++*a.launches;
  return launch_pdl(grad_tokens_kernel, dim3((unsigned)((a.n + 255) / 256)), 256, 0, a.st, p);
}

cudaError_t grad_targets(const HeadGrad& a, const SoftmaxTokens& t) {
  ++*a.launches;
  return launch_pdl(grad_targets_kernel, dim3((unsigned)((a.n + 255) / 256)), 256, 0, a.st, tokens_params(a, t));
}

cudaError_t grad_product(const HeadGrad& a, const float* dnll, uint16_t* dH) {
  const archead_head& h = *a.head;
  const GradPlan g = grad_plan(h, a.n);
  const GradParts b = grad_parts(a, g);
  int gs = 0;
  while ((1 << gs) < h.g) ++gs;
  const GradParams p = {h, b.img, b.cs, b.part, a.n, g.dp, g.nunits, g.nimg, g.ntt, g.ntiles, g.slabs, gs, b.fimg, g.fcols, a.err};
  cudaError_t e;
  if (g.warp) {
    e = launch_grad_warp({h, b.img, b.cs, b.fimg, b.part, a.n, g.dp, g.nunits, g.it, g.fcols, g.slabs, gs, a.err}, a.st);
  } else if (g.mt == 2) {
    e = launch_grad_it<128, 2>(p, a.st);
  } else {
    switch (g.it) {
      case 16: e = launch_grad_it<16, 1>(p, a.st); break;
      case 32: e = launch_grad_it<32, 1>(p, a.st); break;
      case 64: e = launch_grad_it<64, 1>(p, a.st); break;
      default: e = launch_grad_it<128, 1>(p, a.st); break;
    }
  }
  if (e != cudaSuccess) return e;
  const FinishParams fp = {h, b.part, a.n, g.dp, g.slabs, b.texp, dnll, reinterpret_cast<__nv_bfloat16*>(dH)};
  *a.launches += 2;
  // 64 tokens per block share b, where such blocks are many: they hold u in shared memory and have few
  // threads, so with 16 tokens more loads are in flight.  A call at V = 32000, D = 4096 in blocks of 16 and of
  // 64: 128 ranks N = 1500 (768 blocks of 64) 495 and 543 us, N = 2048 (1024) 614 and 596, N = 4096 1241 and 1188; 256 ranks
  // N = 600 219 and 324 (V = 20000), N = 4096 1336 and 1436; without ranks N = 600 192 and 190, N = 1024 297 and 285.
  const int ranks = h.r_c + h.r_r;
  const int64_t rounds = (a.n + 63) / 64 * (h.D / 128) / sm_count();
  const int mt = ranks <= 128 && rounds >= (ranks ? 6 : 2) ? 4 : 1;
  const size_t smem = finish_smem(mt, ranks);
  auto kern = mt == 4 ? grad_finish_kernel<4> : grad_finish_kernel<1>;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)((a.n + 16 * mt - 1) / (16 * mt)), (unsigned)(h.D / 128)), finish_threads(mt), smem, a.st, fp);
}

}  // namespace archead
