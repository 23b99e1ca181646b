// Losses on per-token NLLs, each with its gradient (archead_policy_loss and
// archead_preference_loss; formulas in archead.h).
//
// Both are a pass over a few floats per token plus sums over ragged sequences, so device
// memory bounds them when the batch is large and launches when it is small.  Two forms:
//  * small batches (kSmallTokens, kSmallSeqs): one block does everything in one launch, with
//    the sequences' sums in shared memory;
//  * others: the tokens are cut into fixed pieces of 256, one warp each.  A sequence inside a
//    piece is summed by its warp; one that crosses pieces leaves one partial sum per piece
//    (`tail` where it starts, `head` in each later piece), which its readers add in order.
// Sums are FP64 in an order that the sizes alone fix, so equal calls give equal bits.  A
// sequence's slope over the pairs that hold it arrives in any order: it is added in fixed
// point (integer adds commute exactly).
#include <math.h>

#include "tc_common.cuh"

namespace archead {
namespace {

constexpr int kPiece = 256;          // tokens per warp in the sequence sums
constexpr int kTokBlock = 1024;      // tokens per block step in the token kernels
constexpr int kMaxBlocks = 148 * 8;  // blocks of the token kernels (256 threads, 8 per SM)

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the block in a fixed order; thread 0 gets it.  red: one double per warp.
__device__ __forceinline__ double block_sum(double v, double* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = warp_sum(v);
  __syncthreads();  // red of the previous sum has been read
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = 0.0;
  if (warp == 0) v = warp_sum(lane < nw ? red[lane] : 0.0);
  return v;
}

// Offset i of the sequences, taken into [0, N].
__device__ __forceinline__ int64_t seq_at(const int32_t* cu, int64_t i, int64_t N) {
  const int64_t c = __ldg(cu + i);
  return c < 0 ? 0 : (c > N ? N : c);
}

// The sequence among [lo, hi) that holds token t (empty ones hold none), or -1.
__device__ __forceinline__ int64_t seq_of(const int32_t* cu, int64_t lo, int64_t hi, int64_t N,
                                          int64_t t) {
  // largest i in [lo, hi) with cu[i] <= t
  if (hi <= lo || seq_at(cu, lo, N) > t) return -1;
  int64_t a = lo, b = hi;  // cu[a] <= t, cu[b] > t or b == hi
  while (b - a > 1) {
    const int64_t m = (a + b) >> 1;
    if (seq_at(cu, m, N) <= t) a = m;
    else b = m;
  }
  return t < seq_at(cu, a + 1, N) ? a : -1;
}

__device__ __forceinline__ bool seq_bad(const int32_t* cu, int64_t i, int64_t N) {
  const int64_t a = __ldg(cu + i), b = __ldg(cu + i + 1);
  return a < 0 || b < a || b > N;
}

// ---- sequence sums ----------------------------------------------------------------------
// Per token a weight and a value; per sequence their sums.
struct Pair2 {
  double w, x;
};

struct SeqSums {
  Pair2* whole;  // B: sequences inside one piece
  Pair2* head;   // per piece: the sequence that began before it
  Pair2* tail;   // per piece: the sequence that begins in it and goes on
};

// x = w (nll_ref - nll) with nll given (preference scores); nll == nullptr: weights alone.
__device__ __forceinline__ Pair2 token_pair(const float* nll, const float* ref, const float* w,
                                            int64_t t) {
  Pair2 p;
  p.w = w ? (double)__ldg(w + t) : 1.0;
  p.x = 0.0;
  if (nll && p.w != 0.0)
    p.x = p.w * ((ref ? (double)__ldg(ref + t) : 0.0) - (double)__ldg(nll + t));
  return p;
}

__global__ void __launch_bounds__(256) seq_sums_kernel(const float* __restrict__ nll,
                                                       const float* __restrict__ ref,
                                                       const float* __restrict__ w,
                                                       const int32_t* __restrict__ cu, int64_t N,
                                                       int64_t B, SeqSums out,
                                                       unsigned long long* zero, int64_t nzero,
                                                       unsigned* err) {
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int64_t gtid = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int64_t gsize = (int64_t)gridDim.x * blockDim.x;
  bool bad = false;
  for (int64_t i = gtid; i < B; i += gsize) bad |= seq_bad(cu, i, N);
  if (bad) atomicOr(err, kErrSegment);
  for (int64_t i = gtid; i < nzero; i += gsize) zero[i] = 0ull;
  const int64_t c = gtid >> 5;  // this warp's piece
  const int64_t t0 = c * kPiece;
  if (t0 >= N) return;
  const int64_t t1 = t0 + kPiece < N ? t0 + kPiece : N;
  Pair2 v[kPiece / 32];
#pragma unroll
  for (int k = 0; k < kPiece / 32; ++k) {
    const int64_t t = t0 + 32 * k + lane;
    v[k] = t < t1 ? token_pair(nll, ref, w, t) : Pair2{0.0, 0.0};
  }
  int64_t pos = t0;
  const int64_t first = seq_at(cu, 0, N);
  if (pos < first) pos = first;  // tokens before the first sequence
  int64_t s = -1;
  while (pos < t1) {
    // the next sequence is usually the one after; empty ones are skipped by a search
    int64_t n = s >= 0 && s + 1 < B ? s + 1 : -1;
    if (n >= 0 && !(seq_at(cu, n, N) <= pos && pos < seq_at(cu, n + 1, N))) n = -1;
    s = n >= 0 ? n : seq_of(cu, 0, B, N, pos);
    if (s < 0) break;  // behind the last sequence
    const int64_t b0 = seq_at(cu, s, N), b1 = seq_at(cu, s + 1, N);
    const int64_t hi = b1 < t1 ? b1 : t1;
    Pair2 a = {0.0, 0.0};
#pragma unroll
    for (int k = 0; k < kPiece / 32; ++k) {
      const int64_t t = t0 + 32 * k + lane;
      if (t >= pos && t < hi) {
        a.w += v[k].w;
        a.x += v[k].x;
      }
    }
    a.w = warp_sum(a.w);
    if (nll) a.x = warp_sum(a.x);
    if (lane == 0) {
      Pair2* dst = b0 < t0 ? out.head + c : (b1 > t1 ? out.tail + c : out.whole + s);
      *dst = a;
    }
    pos = hi;
  }
}

// The sums of sequence s, by a whole warp (every lane gets them).
__device__ __forceinline__ Pair2 seq_total(const SeqSums& q, const int32_t* cu, int64_t s,
                                           int64_t N) {
  const int64_t b0 = seq_at(cu, s, N), b1 = seq_at(cu, s + 1, N);
  if (b1 <= b0) return {0.0, 0.0};
  const int64_t c0 = b0 / kPiece, c1 = (b1 - 1) / kPiece;
  if (c0 == c1) return q.whole[s];
  Pair2 a = {0.0, 0.0};
  for (int64_t c = c0 + 1 + (threadIdx.x & 31); c <= c1; c += 32) {
    const Pair2 h = q.head[c];
    a.w += h.w;
    a.x += h.x;
  }
  a.w = warp_sum(a.w);
  a.x = warp_sum(a.x);
  const Pair2 t = q.tail[c0];
  return {t.w + a.w, t.x + a.x};
}

// ---- policy loss ------------------------------------------------------------------------
struct PolicyConst {
  double log_hi, log_lo;  // log(1 + clip_high), log(1 - clip_low)
  double hi, lo;          // 1 + clip_high, 1 - clip_low
  double kl_coef;
};

struct PolicyTok {
  double sur, kl, clipped, grad;
};

// exp(z) - 1 - z: its Taylor series near 0, where the difference cancels (the first term left
// out is below 5e-8 of the sum at |z| = 1/2).
__device__ __forceinline__ float kl_term(float z, float em1) {
  if (fabsf(z) >= 0.5f) return em1 - z;
  float p = fmaf(z, 1.f / 8, 1.f);
  p = fmaf(z * (1.f / 7), p, 1.f);
  p = fmaf(z * (1.f / 6), p, 1.f);
  p = fmaf(z * (1.f / 5), p, 1.f);
  p = fmaf(z * (1.f / 4), p, 1.f);
  p = fmaf(z * (1.f / 3), p, 1.f);
  return 0.5f * z * z * p;
}

// One token: r = exp(x), x = nll_old - nll.  Which side of the clip border it lies on is
// decided by the exact difference of the two FP32 values against log(1 +- clip) in FP64.
__device__ __forceinline__ PolicyTok policy_token(float nll, float old, float A, bool has_ref,
                                                  float ref, const PolicyConst& k) {
  const double x = (double)old - (double)nll;
  PolicyTok o = {0.0, 0.0, 0.0, 0.0};
  if (A != 0.f) {  // (0 times an infinite ratio is 0 here)
    if ((A > 0.f && x > k.log_hi) || (A < 0.f && x < k.log_lo)) {
      o.sur = -(A > 0.f ? k.hi : k.lo) * (double)A;
      o.clipped = 1.0;
    } else {
      o.grad = (double)(expf((float)x) * A);
      o.sur = -o.grad;
    }
  }
  if (has_ref) {
    const float z = nll - ref, em1 = expm1f(z);
    o.kl = (double)kl_term(z, em1);
    o.grad += k.kl_coef * (double)em1;
  }
  return o;
}

// Per-sequence scale 1 / sum w (0 for a sequence without weight) and how many sequences
// have weight, one warp per sequence.  Without weights the sum is the length.
__global__ void __launch_bounds__(256) policy_seq_kernel(SeqSums q, const float* w,
                                                         const int32_t* __restrict__ cu,
                                                         int64_t N, int64_t B,
                                                         double* __restrict__ inv,
                                                         unsigned* __restrict__ active,
                                                         unsigned* err) {
  allow_dependent_launch();
  grid_dependency_wait();
  __shared__ unsigned cnt[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned n = 0;
  bool bad = false;
  for (int64_t s = blockIdx.x * 8ll + warp; s < B; s += gridDim.x * 8ll) {
    double t;
    if (w) {
      t = seq_total(q, cu, s, N).w;
    } else {
      bad |= seq_bad(cu, s, N);
      const int64_t len = seq_at(cu, s + 1, N) - seq_at(cu, s, N);
      t = len > 0 ? (double)len : 0.0;
    }
    if (lane == 0) inv[s] = t > 0.0 ? 1.0 / t : 0.0;
    n += t > 0.0;
  }
  if (bad) atomicOr(err, kErrSegment);
  if (lane == 0) cnt[warp] = n;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned a = 0;
    for (int i = 0; i < 8; ++i) a += cnt[i];
    active[blockIdx.x] = a;
  }
}

// Sum of the weights of the tokens inside sequences (of all tokens without cu): per block.
__global__ void __launch_bounds__(256) policy_weight_kernel(const float* __restrict__ w,
                                                            const int32_t* __restrict__ cu,
                                                            int64_t N, int64_t B,
                                                            double* __restrict__ part,
                                                            unsigned* err) {
  allow_dependent_launch();
  __shared__ double red[8];
  const int64_t gtid = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int64_t gsize = (int64_t)gridDim.x * blockDim.x;
  int64_t lo = 0, hi = N;
  if (cu) {
    bool bad = false;
    for (int64_t i = gtid; i < B; i += gsize) bad |= seq_bad(cu, i, N);
    if (bad) atomicOr(err, kErrSegment);
    lo = B > 0 ? seq_at(cu, 0, N) : N;
    hi = seq_at(cu, B, N);
  }
  double a = 0.0;
  if (w)
    for (int64_t t = lo + gtid; t < hi; t += gsize) a += (double)__ldg(w + t);
  else if (gtid == 0 && hi > lo)
    a = (double)(hi - lo);
  a = block_sum(a, red);
  if (threadIdx.x == 0) part[blockIdx.x] = a;
}

// The tokens: gradient, and the block's sums of surrogate, KL term and clipped weight.
__global__ void __launch_bounds__(256) policy_token_kernel(
    PolicyArgs a, PolicyConst k, const double* __restrict__ inv, const unsigned* active,
    int nactive, const double* wpart, int nwpart, double* __restrict__ part, unsigned* err) {
  allow_dependent_launch();
  grid_dependency_wait();
  __shared__ double red[8];
  __shared__ double scale_s;
  __shared__ int64_t seq_lo, seq_hi;
  // the common factor: 1 / sum w, 1 / (sequences with weight), or 1
  double t = 0.0;
  if (a.reduction == ARCHEAD_REDUCE_TOKEN) {
    for (int i = threadIdx.x; i < nwpart; i += 256) t += wpart[i];
  } else if (a.reduction == ARCHEAD_REDUCE_SEQUENCE) {
    for (int i = threadIdx.x; i < nactive; i += 256) t += (double)active[i];
  } else if (threadIdx.x == 0) {
    t = 1.0;
  }
  t = block_sum(t, red);
  if (threadIdx.x == 0) scale_s = t > 0.0 ? 1.0 / t : 0.0;
  __syncthreads();
  const double scale = scale_s;
  if (a.cu && a.reduction == ARCHEAD_REDUCE_SUM) {  // nothing before this kernel looked
    bool bad = false;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < a.B; i += gridDim.x * 256ll)
      bad |= seq_bad(a.cu, i, a.N);
    if (bad) atomicOr(err, kErrSegment);
  }
  double sur = 0.0, kl = 0.0, clipped = 0.0;
  const bool need_seq = a.adv_per_seq || a.reduction == ARCHEAD_REDUCE_SEQUENCE;
  const int64_t first = a.cu ? (a.B > 0 ? seq_at(a.cu, 0, a.N) : a.N) : 0;
  const int64_t last = a.cu ? seq_at(a.cu, a.B, a.N) : a.N;
  for (int64_t c0 = (int64_t)blockIdx.x * kTokBlock; c0 < a.N; c0 += (int64_t)gridDim.x * kTokBlock) {
    if (need_seq) {  // the sequences that this step's tokens can lie in
      __syncthreads();
      if (threadIdx.x < 2) {
        int64_t x = threadIdx.x ? c0 + kTokBlock - 1 : c0;
        if (x >= last) x = last - 1;
        if (x < first) x = first;
        const int64_t s = last > first ? seq_of(a.cu, 0, a.B, a.N, x) : -1;
        if (threadIdx.x) seq_hi = s < 0 ? a.B : s + 1;
        else seq_lo = s < 0 ? 0 : s;
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kTokBlock / 256; ++j) {
      const int64_t n = c0 + 256 * j + threadIdx.x;
      if (n >= a.N) break;
      double w = n >= first && n < last ? (a.w ? (double)__ldg(a.w + n) : 1.0) : 0.0;
      int64_t s = 0;
      if (need_seq && w != 0.0) {
        s = seq_of(a.cu, seq_lo, seq_hi, a.N, n);
        if (s < 0) w = 0.0;  // only where the offsets are out of order
      }
      float g = 0.f;
      if (w != 0.0) {
        const float A = __ldg(a.adv + (a.adv_per_seq ? s : n));
        const PolicyTok o = policy_token(__ldg(a.nll + n), __ldg(a.nll_old + n), A,
                                         a.nll_ref != nullptr,
                                         a.nll_ref ? __ldg(a.nll_ref + n) : 0.f, k);
        w *= scale;
        if (a.reduction == ARCHEAD_REDUCE_SEQUENCE) w *= inv[s];
        sur += w * o.sur;
        kl += w * o.kl;
        clipped += w * o.clipped;
        g = (float)(w * o.grad);
      }
      a.dnll[n] = g;
    }
  }
  const double s0 = block_sum(sur, red), s1 = block_sum(kl, red), s2 = block_sum(clipped, red);
  if (threadIdx.x == 0) {
    part[3 * blockIdx.x] = s0;
    part[3 * blockIdx.x + 1] = s1;
    part[3 * blockIdx.x + 2] = s2;
  }
}

__device__ __forceinline__ void policy_stats(float* stats, double sur, double kl,
                                             double clipped, double kl_coef) {
  stats[0] = (float)(kl_coef != 0.0 ? sur + kl_coef * kl : sur);
  stats[1] = (float)sur;
  stats[2] = (float)kl;
  stats[3] = (float)clipped;
}

__global__ void __launch_bounds__(256) policy_final_kernel(const double* __restrict__ part, int n,
                                                           double kl_coef, float* stats) {
  grid_dependency_wait();
  __shared__ double red[8];
  double s[3] = {0.0, 0.0, 0.0};
  for (int i = threadIdx.x; i < n; i += 256)
#pragma unroll
    for (int j = 0; j < 3; ++j) s[j] += part[3 * i + j];
#pragma unroll
  for (int j = 0; j < 3; ++j) s[j] = block_sum(s[j], red);
  if (threadIdx.x == 0) policy_stats(stats, s[0], s[1], s[2], kl_coef);
}

PolicyConst policy_const(const PolicyArgs& a) {
  return {log1p(a.clip_high), log1p(-a.clip_low), 1.0 + a.clip_high, 1.0 - a.clip_low, a.kl_coef};
}

int token_blocks(int64_t N) {
  int64_t b = (N + kTokBlock - 1) / kTokBlock;
  return (int)(b < 1 ? 1 : (b > kMaxBlocks ? kMaxBlocks : b));
}
int seq_blocks(int64_t B) {
  int64_t b = (B + 7) / 8;
  return (int)(b < 1 ? 1 : (b > kMaxBlocks ? kMaxBlocks : b));
}
int64_t piece_count(int64_t N) { return (N + kPiece - 1) / kPiece; }

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
size_t seq_sum_bytes(int64_t N, int64_t B) {
  return up256((size_t)B * sizeof(Pair2)) + 2 * up256((size_t)piece_count(N) * sizeof(Pair2));
}
SeqSums carve_seq_sums(char* b, int64_t N, int64_t B) {
  SeqSums q;
  q.whole = reinterpret_cast<Pair2*>(b);
  q.head = reinterpret_cast<Pair2*>(b + up256((size_t)B * sizeof(Pair2)));
  q.tail = reinterpret_cast<Pair2*>(reinterpret_cast<char*>(q.head) +
                                    up256((size_t)piece_count(N) * sizeof(Pair2)));
  return q;
}

// A launch that may start while the previous kernel of the stream runs (its kernel waits for
// it before reading its results).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), int64_t grid, int threads, cudaStream_t st,
                         A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// ---- preference loss --------------------------------------------------------------------
// A sequence's slope dL/df over its pairs, in fixed point: four signed 64-bit limbs, limb k
// of weight 2^(32 k - 96), so sums up to 2^31 pairs keep every bit above 2^-96 (of the unit
// that the host chooses, about the largest slope of an ordinary pair) and integer adds make
// the result independent of their order.  A slope that is not finite, or above 2^31 units,
// counts in a fifth word and makes the sequence's slope NaN.
constexpr int kLimbs = 5;

__device__ __forceinline__ void slope_add(unsigned long long* acc, double v) {
  if (!(fabs(v) < 2147483648.0)) {
    atomicAdd(acc + 4, 1ull);
    return;
  }
#pragma unroll
  for (int k = 3; k >= 0; --k) {
    const long long d = (long long)v;  // toward zero
    if (d) atomicAdd(acc + k, (unsigned long long)d);
    v = (v - (double)d) * 4294967296.0;  // exact: a power of two and the fraction's bits
  }
}

__device__ __forceinline__ double slope_value(const unsigned long long* acc) {
  if (acc[4]) return __longlong_as_double(0x7ff8000000000000ll);
  double v = 0.0, unit = 1.0 / 4294967296.0 / 4294967296.0 / 4294967296.0;
#pragma unroll
  for (int k = 0; k < 4; ++k, unit *= 4294967296.0) v += (double)(long long)acc[k] * unit;
  return v;
}

struct PrefConst {
  double beta, smoothing, margin, unit;  // slopes are counted in units of `unit`
  int kind;
};

// loss and its slope by f_a - f_b
__device__ __forceinline__ void pref_pair(double gap, const PrefConst& k, double* loss,
                                          double* slope) {
  const double m = k.beta * gap - k.margin;
  if (k.kind == ARCHEAD_PREF_SIGMOID) {
    // -log sigma(m) = log(1 + e^-|m|) + max(-m, 0), and one of the two sigmas is 1 / (1 + e)
    const double e = exp(-fabs(m)), l = log1p(e), big = 1.0 / (1.0 + e), small = e / (1.0 + e);
    const double up = m >= 0 ? big : small, down = m >= 0 ? small : big;  // sigma(m), sigma(-m)
    *loss = l + (m >= 0 ? k.smoothing * m : -(1.0 - k.smoothing) * m);
    *slope = k.beta * (k.smoothing * up - (1.0 - k.smoothing) * down);
    if (m != m) *loss = *slope = m;
  } else if (k.kind == ARCHEAD_PREF_HINGE) {
    *loss = m < 1.0 ? 1.0 - m : (m != m ? m : 0.0);
    *slope = m < 1.0 ? -k.beta : (m != m ? m : 0.0);
  } else {
    const double d = gap - k.margin - 0.5 / k.beta;
    *loss = d * d;
    *slope = 2.0 * d;
  }
}

__device__ __forceinline__ double score_of(const Pair2& t, int average) {
  return average ? (t.w > 0.0 ? t.x / t.w : 0.0) : t.x;
}

// One warp per pair: its loss and rewards, its slope into both sequences' accumulators, and
// the block's sum of losses.
__global__ void __launch_bounds__(256) pref_pair_kernel(PreferenceArgs a, PrefConst k, SeqSums q,
                                                        unsigned long long* acc, double* part,
                                                        unsigned* err) {
  allow_dependent_launch();
  grid_dependency_wait();
  __shared__ double red[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double sum = 0.0;
  for (int64_t p = blockIdx.x * 8ll + warp; p < a.P; p += gridDim.x * 8ll) {
    const int64_t ia = __ldg(a.pairs + 2 * p), ib = __ldg(a.pairs + 2 * p + 1);
    double loss, slope = 0.0, fa, fb;
    if (ia < 0 || ia >= a.B || ib < 0 || ib >= a.B) {
      loss = fa = fb = __longlong_as_double(0x7ff8000000000000ll);
      if (lane == 0) atomicOr(err, kErrSegment);
    } else {
      fa = score_of(seq_total(q, a.cu, ia, a.N), a.average);
      fb = score_of(seq_total(q, a.cu, ib, a.N), a.average);
      pref_pair(fa - fb, k, &loss, &slope);
      if (lane == 0) {
        slope_add(acc + ia * kLimbs, slope * k.unit);
        slope_add(acc + ib * kLimbs, -slope * k.unit);
      }
    }
    if (lane == 0) {
      a.pair_loss[p] = (float)loss;
      a.rewards[2 * p] = (float)(k.beta * fa);
      a.rewards[2 * p + 1] = (float)(k.beta * fb);
      sum += loss;
    }
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// dnll[n] = -w [/ sum w] slope(sequence) / P, one warp per piece as in seq_sums_kernel; block
// 0 also adds the losses.
__global__ void __launch_bounds__(256) pref_token_kernel(PreferenceArgs a, PrefConst k, SeqSums q,
                                                         const unsigned long long* acc,
                                                         const double* part, int npart) {
  grid_dependency_wait();
  __shared__ double red[8];
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) {
    double s = 0.0;
    for (int i = threadIdx.x; i < npart; i += 256) s += part[i];
    s = block_sum(s, red);
    if (threadIdx.x == 0) a.loss[0] = a.P ? (float)(s / (double)a.P) : 0.f;
  }
  const int64_t c = (blockIdx.x * 256ll + threadIdx.x) >> 5;
  const int64_t t0 = c * kPiece;
  if (t0 >= a.N) return;
  const int64_t t1 = t0 + kPiece < a.N ? t0 + kPiece : a.N;
  float w[kPiece / 32], g[kPiece / 32];
#pragma unroll
  for (int i = 0; i < kPiece / 32; ++i) {
    const int64_t t = t0 + 32 * i + lane;
    w[i] = t < t1 ? (a.w ? __ldg(a.w + t) : 1.f) : 0.f;
    g[i] = 0.f;
  }
  const double per_pair = a.P ? 1.0 / (k.unit * (double)a.P) : 0.0;
  int64_t pos = t0;
  const int64_t first = seq_at(a.cu, 0, a.N);
  if (pos < first) pos = first;
  int64_t s = -1;
  while (pos < t1) {
    int64_t n = s >= 0 && s + 1 < a.B ? s + 1 : -1;
    if (n >= 0 && !(seq_at(a.cu, n, a.N) <= pos && pos < seq_at(a.cu, n + 1, a.N))) n = -1;
    s = n >= 0 ? n : seq_of(a.cu, 0, a.B, a.N, pos);
    if (s < 0) break;
    const int64_t b1 = seq_at(a.cu, s + 1, a.N);
    const int64_t hi = b1 < t1 ? b1 : t1;
    double coef = -slope_value(acc + s * kLimbs) * per_pair;
    if (a.average) {
      const double t = seq_total(q, a.cu, s, a.N).w;
      coef = t > 0.0 ? coef / t : 0.0;
    }
#pragma unroll
    for (int i = 0; i < kPiece / 32; ++i) {
      const int64_t t = t0 + 32 * i + lane;
      if (t >= pos && t < hi && w[i] != 0.f) g[i] = (float)(coef * (double)w[i]);
    }
    pos = hi;
  }
#pragma unroll
  for (int i = 0; i < kPiece / 32; ++i) {
    const int64_t t = t0 + 32 * i + lane;
    if (t < t1) a.dnll[t] = g[i];
  }
}

PrefConst pref_const(const PreferenceArgs& a) {
  PrefConst k = {a.beta, a.smoothing, a.margin, 1.0, a.kind};
  // the largest slope of an ordinary pair: beta, or 1 / beta for ipo
  k.unit = ldexp(1.0, -ilogb(a.kind == ARCHEAD_PREF_IPO ? fmax(1.0, 1.0 / a.beta) : a.beta));
  return k;
}

}  // namespace

size_t policy_scratch_bytes(const PolicyArgs& a) {
  size_t b = 3 * 8 * kMaxBlocks + up256(8 * kMaxBlocks) + up256(4 * kMaxBlocks);
  if (a.reduction == ARCHEAD_REDUCE_SEQUENCE)
    b += up256((size_t)a.B * 8) + (a.w ? seq_sum_bytes(a.N, a.B) : 0);
  return b;
}

cudaError_t launch_policy_loss(const PolicyArgs& a, void* scratch, unsigned* err,
                               cudaStream_t st, int* launches) {
  char* b = static_cast<char*>(scratch);
  const PolicyConst k = policy_const(a);
  double* part = reinterpret_cast<double*>(b);
  b += 3 * 8 * kMaxBlocks;
  double* wpart = reinterpret_cast<double*>(b);
  b += up256(8 * kMaxBlocks);
  unsigned* active = reinterpret_cast<unsigned*>(b);
  b += up256(4 * kMaxBlocks);
  const int nb = token_blocks(a.N);
  int nwp = 0, nact = 0;
  double* inv = nullptr;
  if (a.reduction == ARCHEAD_REDUCE_TOKEN) {
    nwp = nb;
    policy_weight_kernel<<<nb, 256, 0, st>>>(a.w, a.cu, a.N, a.B, wpart, err);
    ++*launches;
  } else if (a.reduction == ARCHEAD_REDUCE_SEQUENCE) {
    inv = reinterpret_cast<double*>(b);
    b += up256((size_t)a.B * 8);
    SeqSums q = {};
    if (a.w) {
      q = carve_seq_sums(b, a.N, a.B);
      const int64_t blocks = (piece_count(a.N) + 7) / 8;
      seq_sums_kernel<<<(unsigned)(blocks < 1 ? 1 : blocks), 256, 0, st>>>(
          nullptr, nullptr, a.w, a.cu, a.N, a.B, q, nullptr, 0, err);
      ++*launches;
    }
    nact = seq_blocks(a.B);
    const cudaError_t e = launch_after(policy_seq_kernel, nact, 256, st, q, a.w, a.cu, a.N, a.B,
                                       inv, active, err);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  cudaError_t e = launch_after(policy_token_kernel, nb, 256, st, a, k, inv, active, nact, wpart,
                               nwp, part, err);
  if (e != cudaSuccess) return e;
  e = launch_after(policy_final_kernel, 1, 256, st, part, nb, a.kl_coef, a.stats);
  *launches += 2;
  return e;
}

size_t preference_scratch_bytes(const PreferenceArgs& a) {
  return up256(8 * kMaxBlocks) + up256((size_t)a.B * kLimbs * 8) + seq_sum_bytes(a.N, a.B);
}

cudaError_t launch_preference_loss(const PreferenceArgs& a, void* scratch, unsigned* err,
                                   cudaStream_t st, int* launches) {
  char* b = static_cast<char*>(scratch);
  const PrefConst k = pref_const(a);
  double* part = reinterpret_cast<double*>(b);
  b += up256(8 * kMaxBlocks);
  unsigned long long* acc = reinterpret_cast<unsigned long long*>(b);
  b += up256((size_t)a.B * kLimbs * 8);
  const SeqSums q = carve_seq_sums(b, a.N, a.B);
  int64_t pb = (piece_count(a.N) + 7) / 8;
  if (pb < 1) pb = 1;
  seq_sums_kernel<<<(unsigned)pb, 256, 0, st>>>(a.nll, a.nll_ref, a.w, a.cu, a.N, a.B, q, acc,
                                               a.B * kLimbs, err);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int np = seq_blocks(a.P);
  e = launch_after(pref_pair_kernel, np, 256, st, a, k, q, acc, part, err);
  if (e != cudaSuccess) return e;
  e = launch_after(pref_token_kernel, pb, 256, st, a, k, q, acc, part, np);
  *launches += 3;
  return e;
}

}  // namespace archead
