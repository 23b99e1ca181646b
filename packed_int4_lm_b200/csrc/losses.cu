// Losses on per-token NLLs, each with its gradient (archead_policy_loss and
// archead_preference_loss; formulas in archead.h).
//
// Both are a pass over a few floats per token plus sums over ragged sequences.  The tokens are cut
// into pieces of 256: a lane holds eight tokens of a piece, two 16-byte loads per array where the
// arrays are aligned to it, and a warp walks the sequences that lie in its pieces (adjacent ones, so
// that the first sequence is searched for once, 32 probes a step).  A sequence inside a piece is
// summed by its warp, a short one among others by a lane; one that crosses pieces leaves one partial
// sum per piece (`tail` where it starts, `head` in each later piece), which its readers add in
// order.  The steps are device functions:
//  * small batches (at most 32 pieces) run them in one block, in one launch, with the sequences' sums in
//    shared memory (7 sequences of 40 tokens: 13 us a call against 22 us for the chain, most of it
//    the host's);
//  * others in a chain of launches, each waiting for the one before (8192 sequences, 4.2 M tokens:
//    policy 45 us, preference 36 us; their arrays alone take 18 and 10 us at the measured copy rate.
//    Latency bounds them: one by one the launches take 14, 7, 29 and 6, and 17, 11 and 15 us, with issue
//    slots used to 57 and 47 % at most and DRAM to 38 %).
// Sums are FP64 in an order that the sizes alone fix, so equal calls give equal bits.  A
// sequence's slope over the pairs that hold it arrives in any order: it is added in fixed
// point (integer adds commute exactly).
#include <math.h>

#include <type_traits>

#include "tc_common.cuh"

namespace archead {
namespace {

constexpr int kPer = 8, kPiece = 32 * kPer;  // tokens per lane, per warp
constexpr int kMaxBlocks = 148 * 4;          // blocks of a launch: what runs at once, so that a
                                             // warp's pieces lie side by side
constexpr int kSmallPieces = 32;             // what one block takes, one piece per warp
constexpr int kSmallSeqs = 256, kSmallPairs = 192;  // (more of them take longer in one block than the
                                                    // chain: 256 sequences, 256 pairs 30 against 24 us)

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the block in a fixed order; warp 0 gets it.  red: one double per warp.
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

// ---- sequences --------------------------------------------------------------------------
struct Seqs {
  const int32_t* cu;  // B + 1 offsets, or nullptr: one sequence of all tokens
  int N, B;
};

// Offset i, taken into [0, N].
__device__ __forceinline__ int seq_at(const Seqs& q, int64_t i) {
  const int c = __ldg(q.cu + i);
  return c < 0 ? 0 : (c > q.N ? q.N : c);
}
__device__ __forceinline__ bool seq_bad(const Seqs& q, int i) {
  const int a = __ldg(q.cu + i), b = __ldg(q.cu + i + 1);
  return a < 0 || b < a || b > q.N;
}
// Reports offsets that fall or leave [0, N], shared out over `size` threads.
__device__ __forceinline__ void check_seqs(const Seqs& q, int64_t tid, int64_t size, unsigned* err) {
  if (!q.cu) return;
  bool bad = q.B == 0 && tid == 0 && (__ldg(q.cu) < 0 || __ldg(q.cu) > q.N);
  for (int64_t i = tid; i < q.B; i += size) bad |= seq_bad(q, (int)i);
  if (bad) atomicOr(err, kErrSegment);
}

// The last sequence that begins at or before token t, by a whole warp; -1 if none does.  (Where
// the offsets are out of order it is some index in range.)
__device__ __forceinline__ int warp_seq_of(const Seqs& q, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = q.B;  // of lo .. lo + n - 1 the first few begin at or before t
  while (n > 32) {
    const int step = ((n - 1) >> 5) + 1;
    const int64_t i = (lane + 1ll) * step - 1;  // (passes 2^31 with the most sequences)
    const bool in = i < n && seq_at(q, lo + i) <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, in)) * step;
    lo += c;
    n = n - c < step ? n - c : step;
  }
  const bool in = lane < n && seq_at(q, lo + lane) <= t;
  return lo + __popc(__ballot_sync(0xffffffffu, in)) - 1;
}

// Walks the sequences along adjacent pieces, one warp: window(i) lets each lane load what belongs
// to sequence i (32 sequences at a time), and piece(t0, t1, f) calls f(j, s, lo, hi, b0, b1) with
// the whole warp for the tokens [lo, hi) of sequence s = [b0, b1), whose window data lane j holds.
// Short sequences inside the piece are taken several at once, by many(s, lo, hi, b0, b1, mine): lane
// j has sequence s + j = [b0, b1) if it is one of them (mine), and [lo, hi) are the tokens of all (6500
// sequences of one token, preference: 144 -> 33 us; 8192 of 512 tokens 31 -> 32 us).
template <typename W>
struct Walker {
  const Seqs q;
  W window;
  unsigned s = 0;  // the window's first sequence (unsigned: windows pass the last sequence, which may be 2^31 - 3)
  int j = 0, b0 = 0, end = 0;  // the current one in it, its start

  __device__ __forceinline__ void load() {
    const unsigned i = s + (threadIdx.x & 31);
    end = 0x7fffffff;
    if (i < (unsigned)q.B) {
      end = seq_at(q, i + 1ll);
      window(i);
    }
  }
  __device__ __forceinline__ Walker(const Seqs& seqs, int t0, W w) : q(seqs), window(w) {
    if (q.B == 0) return;
    const int first = warp_seq_of(q, t0);
    s = first < 0 ? 0 : first;
    b0 = seq_at(q, s);
    load();
  }
  template <typename F, typename M>
  __device__ __forceinline__ void piece(int t0, int t1, F f, M many) {
    int pos = t0 < b0 ? b0 : t0;  // (tokens before the first sequence)
    while (pos < t1 && s + j < (unsigned)q.B) {
      const int b1 = __shfl_sync(0xffffffffu, end, j);
      if (pos == b0 && b1 <= t1 && b1 - b0 <= 32) {
        const int before = __shfl_up_sync(0xffffffffu, end, 1), lane = threadIdx.x & 31;
        const int begin = lane == 0 ? b0 : before;
        // (a lane past the last sequence holds no end: t1 may be 0x7fffffff too)
        const bool is_short = s + lane < (unsigned)q.B && end <= t1 && end >= begin && end - begin <= 32;
        const unsigned run = __ballot_sync(0xffffffffu, is_short) >> j;
        const int n = run == 0xffffffffu ? 32 : __ffs(~run) - 1;  // sequences j .. j + n - 1 of the window
        if (n >= 4) {  // (8: 36 against 34 us)
          const int last = __shfl_sync(0xffffffffu, end, j + n - 1);
          const bool mine = lane >= j && lane < j + n;
          many(s, b0, last, mine ? begin : 0, end, mine);
          pos = b0 = last;
          j += n;
          if (j == 32) {
            s += 32;
            j = 0;
            load();
          }
          continue;
        }
      }
      const int hi = b1 < t1 ? b1 : t1;
      if (hi > pos) {
        f(j, s + j, pos, hi, b0, b1);
        pos = hi;
      }
      if (b1 > t1) break;  // goes on in the next piece
      b0 = b1;
      if (++j == 32) {
        s += 32;
        j = 0;
        load();
      }
    }
  }
};

// The lane whose sequence of a window holds token t (b1: the lanes' ends, in order).
__device__ __forceinline__ int lane_of(int b1, int t) {
  int j = 0;
#pragma unroll
  for (int step = 16; step > 0; step >>= 1)
    if (__shfl_sync(0xffffffffu, b1, j + step - 1) <= t) j += step;
  return j;
}

// The lane's i-th token of the piece at t0: two runs of four adjacent ones.
__device__ __forceinline__ int token_at(int t0, int i) {
  return t0 + 128 * (i >> 2) + 4 * (threadIdx.x & 31) + (i & 3);
}
// A piece's values at the lane's tokens; `other` past t1 (and, for p == nullptr, everywhere).
// vec: p is 16-byte aligned.
__device__ __forceinline__ void load_piece(const float* p, int t0, int t1, bool vec, float other, float (&v)[kPer]) {
  if (p && vec && t1 - t0 == kPiece) {
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(p + token_at(t0, i)));
      v[i] = q.x;
      v[i + 1] = q.y;
      v[i + 2] = q.z;
      v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = token_at(t0, i);
      v[i] = p && t < t1 ? __ldg(p + t) : other;
    }
  }
}
__device__ __forceinline__ void store_piece(float* p, int t0, int t1, bool vec, const float (&v)[kPer]) {
  if (vec && t1 - t0 == kPiece) {
#pragma unroll
    for (int i = 0; i < kPer; i += 4)
      __stcs(reinterpret_cast<float4*>(p + token_at(t0, i)), make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (token_at(t0, i) < t1) p[token_at(t0, i)] = v[i];
  }
}
__device__ __forceinline__ bool aligned16(const void* a, const void* b = nullptr, const void* c = nullptr,
                                          const void* d = nullptr, const void* e = nullptr, const void* f = nullptr) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c) |
           reinterpret_cast<uintptr_t>(d) | reinterpret_cast<uintptr_t>(e) | reinterpret_cast<uintptr_t>(f)) & 15) == 0;
}

// Per sequence the sums of a weight and a value.
struct Pair2 {
  double w, x;
};
struct SeqSums {
  Pair2* whole;  // B: sequences inside one piece
  Pair2* head;   // per piece: the sequence that began before it
  Pair2* tail;   // per piece: the sequence that begins in it and goes on
};

// The share of pieces [c, c1): x = w (ref - nll) (kValue), or the weights alone.  A token of
// weight 0 adds nothing, whatever it holds.
template <bool kValue>
__device__ __forceinline__ void sums_pieces(const Seqs& q, const float* nll, const float* ref,
                                            const float* w, int c, int c1, const SeqSums& out) {
  if (c >= c1) return;
  const int lane = threadIdx.x & 31;
  const bool vec = aligned16(nll, ref, w);
  auto none = [](int) {};
  Walker<decltype(none)> walk(q, c * kPiece, none);
  for (; c < c1; ++c) {
    const int t0 = c * kPiece, t1 = q.N - t0 < kPiece ? q.N : t0 + kPiece;
    float wf[kPer], a[kPer], b[kPer];
    load_piece(w, t0, t1, vec, w ? 0.f : 1.f, wf);
    if (kValue) {
      load_piece(nll, t0, t1, vec, 0.f, a);
      load_piece(ref, t0, t1, vec, 0.f, b);
    }
    double x[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      x[k] = kValue && wf[k] != 0.f ? (double)wf[k] * ((double)b[k] - (double)a[k]) : 0.0;
    walk.piece(t0, t1, [&](int, int s, int lo, int hi, int b0, int b1) {
      Pair2 sum = {0.0, 0.0};
      if (hi - lo == kPiece) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          sum.w += (double)wf[k];
          if (kValue) sum.x += x[k];
        }
      } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const bool in = (unsigned)(token_at(t0, k) - lo) < (unsigned)(hi - lo);
          sum.w += in ? (double)wf[k] : 0.0;
          if (kValue) sum.x += in ? x[k] : 0.0;
        }
      }
      sum.w = warp_sum(sum.w);
      if (kValue) sum.x = warp_sum(sum.x);
      if (lane == 0) *(b0 < t0 ? out.head + c : (b1 > t1 ? out.tail + c : out.whole + s)) = sum;
    }, [&](int s, int, int, int b0, int b1, bool mine) {
      Pair2 sum = {0.0, 0.0};
      for (int t = b0; mine && t < b1; ++t) {
        const float f = w ? __ldg(w + t) : 1.f;
        sum.w += (double)f;
        if (kValue && f != 0.f) sum.x += (double)f * ((ref ? (double)__ldg(ref + t) : 0.0) - (double)__ldg(nll + t));
      }
      if (mine) out.whole[s + lane] = sum;
    });
  }
}

// The pieces of this warp when all warps of the grid share `n` pieces out in order.
__device__ __forceinline__ void my_pieces(int n, int* c0, int* c1) {
  const int64_t w = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t all = gridDim.x * (int64_t)(blockDim.x >> 5);
  *c0 = (int)(n * w / all);
  *c1 = (int)(n * (w + 1) / all);
}
__device__ __forceinline__ int pieces_of(int64_t N) { return (int)((N + kPiece - 1) / kPiece); }

// The sums of sequence s, added by `width` adjacent lanes (a power of two; `lane` counts in
// them; all 32 lanes of the warp take part).
__device__ __forceinline__ Pair2 seq_total(const SeqSums& q, const Seqs& sq, int s, int lane, int width) {
  const int b0 = seq_at(sq, s), b1 = seq_at(sq, s + 1);
  const int c0 = b0 / kPiece, c1 = b1 > b0 ? (b1 - 1) / kPiece : c0;
  Pair2 a = {0.0, 0.0};
  for (int c = c0 + 1 + lane; c <= c1; c += width) {
    const Pair2 h = q.head[c];
    a.w += h.w;
    a.x += h.x;
  }
  for (int o = width >> 1; o > 0; o >>= 1) {
    a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
    a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
  }
  if (b1 <= b0) return {0.0, 0.0};
  const Pair2 t = c0 == c1 ? q.whole[s] : q.tail[c0];
  return {t.w + a.w, t.x + a.x};
}

// ---- policy loss ------------------------------------------------------------------------
struct PolicyConst {
  double log_hi, log_lo;     // log(1 + clip_high), log(1 - clip_low)
  float log_hi_f, log_lo_f;  // rounded
  float hi, lo;              // 1 + clip_high, 1 - clip_low
  float kl_coef;
};

struct PolicyTok {
  float sur, kl, grad;  // sur: the surrogate's negative
  bool clipped;
};

// k = e^z - 1 - z and its derivative d = e^z - 1.  Near 0, where the differences cancel, k is z^2 times
// its Taylor series (the first term left out is below 2^-24 of the sum at |z| = 1) and d = z + k.
__device__ __forceinline__ void kl_term(float z, float* k, float* d) {
  float p = 1.f / 479001600;
  p = fmaf(p, z, 1.f / 39916800);
  p = fmaf(p, z, 1.f / 3628800);
  p = fmaf(p, z, 1.f / 362880);
  p = fmaf(p, z, 1.f / 40320);
  p = fmaf(p, z, 1.f / 5040);
  p = fmaf(p, z, 1.f / 720);
  p = fmaf(p, z, 1.f / 120);
  p = fmaf(p, z, 1.f / 24);
  p = fmaf(p, z, 1.f / 6);
  p = fmaf(p, z, 0.5f);
  const bool near = fabsf(z) < 1.f;
  const float up = expf(z) - 1.f, small = z * z * p;
  *k = near ? small : up - z;
  *d = near ? z + small : up;
}

// The side of the clip border is that of the exact difference old - nll against log(1 +- clip).
// Rounding is monotone, so the rounded difference decides unless it equals the rounded border; a piece
// with such a token takes the FP64 difference, which is exact (kExact).  The rest is FP32: the
// difference's rounding moves a ratio by |x| half steps, expf by a few (as ex2 of x log2 e it moved by |x|
// more, and fell to 0 below 2^-126, for 1 us of 46 at 4.2 M tokens).
template <bool kExact>
__device__ __forceinline__ PolicyTok policy_token(float nll, float old, float A, bool has_ref,
                                                  float ref, const PolicyConst& k) {
  const float x = old - nll;
  const bool up = A > 0.f;
  PolicyTok o;
  if (kExact) {
    const double d = (double)old - (double)nll;
    o.clipped = up ? d > k.log_hi : A < 0.f && d < k.log_lo;
  } else {
    o.clipped = up ? x > k.log_hi_f : A < 0.f && x < k.log_lo_f;
  }
  // (0 times an infinite ratio is 0 here; a NaN stays one)
  const float r = A == 0.f ? (x != x ? x : 0.f) : expf(x) * A;
  o.grad = o.clipped ? 0.f : r;
  o.sur = o.clipped ? (up ? k.hi : k.lo) * A : r;
  o.kl = 0.f;
  if (has_ref) {
    float d;
    kl_term(nll - ref, &o.kl, &d);
    // (without a coefficient the term is only reported, and may be infinite)
    if (k.kl_coef != 0.f) o.grad = fmaf(k.kl_coef, d, o.grad);
  }
  return o;
}

// Sums of the loss's parts.
struct PolicySums {
  double sur, kl, clipped;
};

__device__ __forceinline__ Seqs seqs_of(const PolicyArgs& a) { return {a.cu, (int)a.N, (int)a.B}; }

// The tokens of pieces [c, c1): gradients, and the pieces' parts added to `sum` (per lane).  scale
// is the common factor (1 / sum w, 1 / sequences with weight, or 1); inv the sequences' 1 / sum w.
__device__ __forceinline__ void policy_pieces(const PolicyArgs& a, const PolicyConst& k, int c, int c1,
                                              double scale, const double* inv, PolicySums& sum) {
  const Seqs q = seqs_of(a);
  if (c >= c1) return;
  const bool by_seq = a.reduction == ARCHEAD_REDUCE_SEQUENCE, walks = by_seq || a.adv_per_seq;
  const bool vec = aligned16(a.nll, a.nll_old, a.nll_ref, a.adv_per_seq ? nullptr : a.adv, a.w, a.dnll);
  const int first = !q.cu ? 0 : (q.B > 0 ? seq_at(q, 0) : q.N), last = q.cu ? seq_at(q, q.B) : q.N;
  float sc = 0.f, adv = 0.f;  // of the window's sequence
  auto window = [&](int s) {
    sc = (float)(by_seq ? inv[s] * scale : scale);
    if (a.adv_per_seq) adv = __ldg(a.adv + s);
  };
  Walker<decltype(window)> walk(walks ? q : Seqs{nullptr, 0, 0}, c * kPiece, window);
  for (; c < c1; ++c) {
    const int t0 = c * kPiece, t1 = q.N - t0 < kPiece ? q.N : t0 + kPiece;
    float nll[kPer], old[kPer], ref[kPer], A[kPer], f[kPer];
    load_piece(a.nll, t0, t1, vec, 0.f, nll);
    load_piece(a.nll_old, t0, t1, vec, 0.f, old);
    load_piece(a.nll_ref, t0, t1, vec, 0.f, ref);
    load_piece(a.adv_per_seq ? nullptr : a.adv, t0, t1, vec, 0.f, A);
    load_piece(a.w, t0, t1, vec, a.w ? 0.f : 1.f, f);
    if (walks) {
      float g[kPer] = {};  // outside every sequence
      walk.piece(t0, t1, [&](int j, int, int lo, int hi, int, int) {
        const float fs = __shfl_sync(0xffffffffu, sc, j), as = __shfl_sync(0xffffffffu, adv, j);
        if (hi - lo == kPiece) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) g[i] = fs;
          if (a.adv_per_seq) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) A[i] = as;
          }
          return;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const bool in = (unsigned)(token_at(t0, i) - lo) < (unsigned)(hi - lo);
          g[i] = in ? fs : g[i];
          A[i] = in && a.adv_per_seq ? as : A[i];
        }
      }, [&](int, int lo, int hi, int, int b1, bool) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int t = token_at(t0, i), j = lane_of(b1, t);
          const float fs = __shfl_sync(0xffffffffu, sc, j), as = __shfl_sync(0xffffffffu, adv, j);
          const bool in = (unsigned)(t - lo) < (unsigned)(hi - lo);
          g[i] = in ? fs : g[i];
          A[i] = in && a.adv_per_seq ? as : A[i];
        }
      });
#pragma unroll
      for (int i = 0; i < kPer; ++i) f[i] *= g[i];
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int t = token_at(t0, i);
        f[i] = t >= first && t < last ? f[i] * (float)scale : 0.f;
      }
    }
    float g[kPer];
    bool border = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) border |= old[i] - nll[i] == (A[i] > 0.f ? k.log_hi_f : k.log_lo_f);
    auto tokens = [&](auto exact) {  // no branch on the weight: eight chains side by side
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const PolicyTok o = policy_token<decltype(exact)::value>(nll[i], old[i], A[i], a.nll_ref != nullptr, ref[i], k);
        const bool on = f[i] != 0.f;  // a masked token may hold anything
        const double share = (double)f[i];
        sum.sur = fma(share, on ? -(double)o.sur : 0.0, sum.sur);
        sum.kl = fma(share, on ? (double)o.kl : 0.0, sum.kl);
        sum.clipped += on && o.clipped ? share : 0.0;
        g[i] = on ? f[i] * o.grad : 0.f;
      }
    };
    if (__any_sync(0xffffffffu, border)) tokens(std::true_type());
    else tokens(std::false_type());
    store_piece(a.dnll, t0, t1, vec, g);
  }
}

__device__ __forceinline__ void policy_stats(float* stats, const PolicySums& s, double kl_coef) {
  stats[0] = (float)(kl_coef != 0.0 ? s.sur + kl_coef * s.kl : s.sur);
  stats[1] = (float)s.sur;
  stats[2] = (float)s.kl;
  stats[3] = (float)s.clipped;
}

// Weight of the tokens inside sequences (of all without offsets), this thread's share.
__device__ __forceinline__ double weight_share(const PolicyArgs& a, int64_t tid, int64_t size) {
  const Seqs q = seqs_of(a);
  const int lo = !q.cu ? 0 : (q.B > 0 ? seq_at(q, 0) : q.N), hi = q.cu ? seq_at(q, q.B) : q.N;
  if (!a.w) return tid == 0 && hi > lo ? (double)(hi - lo) : 0.0;
  double s = 0.0;
#pragma unroll 4
  for (int64_t t = lo + tid; t < hi; t += size) s += (double)__ldg(a.w + t);
  return s;
}

// 1 / sum w of sequence s (0 without weight), by a group of lanes; without weights the sum is the
// length.
__device__ __forceinline__ double policy_seq_inv(const PolicyArgs& a, const SeqSums& q, int s, int lane, int width) {
  const Seqs sq = seqs_of(a);
  const double t = a.w ? seq_total(q, sq, s, lane, width).w : (double)(seq_at(sq, s + 1) - seq_at(sq, s));
  return t > 0.0 ? 1.0 / t : 0.0;
}

template <bool kValue>
__global__ void __launch_bounds__(256, 4) seq_sums_kernel(const float* __restrict__ nll,
                                                       const float* __restrict__ ref,
                                                       const float* __restrict__ w, Seqs q,
                                                       SeqSums out, unsigned long long* zero,
                                                       int64_t nzero, unsigned* err) {
  allow_dependent_launch();
  const int64_t tid = blockIdx.x * 256ll + threadIdx.x, size = gridDim.x * 256ll;
  int c0, c1;
  my_pieces(pieces_of(q.N), &c0, &c1);
  sums_pieces<kValue>(q, nll, ref, w, c0, c1, out);
  check_seqs(q, tid, size, err);
  for (int64_t i = tid; i < nzero; i += size) zero[i] = 0ull;
}

// Eight lanes per sequence.
__global__ void __launch_bounds__(256) policy_seq_kernel(PolicyArgs a, SeqSums q, double* __restrict__ inv,
                                                         double* __restrict__ active, unsigned* err) {
  allow_dependent_launch();
  grid_dependency_wait();
  __shared__ double red[8];
  double n = 0.0;
  for (int64_t s0 = blockIdx.x * 32ll; s0 < a.B; s0 += gridDim.x * 32ll) {
    const int64_t s = s0 + (threadIdx.x >> 3);
    const double v = policy_seq_inv(a, q, (int)(s < a.B ? s : a.B - 1), threadIdx.x & 7, 8);
    if (s < a.B && (threadIdx.x & 7) == 0) {
      inv[s] = v;
      n += v > 0.0;
    }
  }
  if (!a.w) check_seqs(seqs_of(a), blockIdx.x * 256ll + threadIdx.x, gridDim.x * 256ll, err);
  n = block_sum(n, red);
  if (threadIdx.x == 0) active[blockIdx.x] = n;
}

__global__ void __launch_bounds__(256) policy_weight_kernel(PolicyArgs a, double* __restrict__ part, unsigned* err) {
  allow_dependent_launch();
  __shared__ double red[8];
  const int64_t tid = blockIdx.x * 256ll + threadIdx.x, size = gridDim.x * 256ll;
  const double s = block_sum(weight_share(a, tid, size), red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
  check_seqs(seqs_of(a), tid, size, err);
}

// total: partial sums (n of them) of what the common factor divides by; nullptr: the factor is 1.
__global__ void __launch_bounds__(256, 3) policy_token_kernel(PolicyArgs a, PolicyConst k, const double* inv,
                                                           const double* total, int n, PolicySums* part,
                                                           unsigned* err) {
  allow_dependent_launch();
  grid_dependency_wait();
  __shared__ double red[8];
  double scale = 1.0;
  if (total) {  // every warp for itself: no barrier before its loads
    double t = 0.0;
    for (int i = threadIdx.x & 31; i < n; i += 32) t += total[i];
    t = warp_sum(t);
    scale = t > 0.0 ? 1.0 / t : 0.0;
  } else {
    check_seqs(seqs_of(a), blockIdx.x * 256ll + threadIdx.x, gridDim.x * 256ll, err);
  }
  PolicySums s = {0.0, 0.0, 0.0};
  int c0, c1;
  my_pieces(pieces_of(a.N), &c0, &c1);
  policy_pieces(a, k, c0, c1, scale, inv, s);
  s.sur = block_sum(s.sur, red);
  s.kl = block_sum(s.kl, red);
  s.clipped = block_sum(s.clipped, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ void __launch_bounds__(256) policy_final_kernel(const PolicySums* __restrict__ part, int n,
                                                           double kl_coef, float* stats) {
  grid_dependency_wait();
  __shared__ double red[8];
  PolicySums s = {0.0, 0.0, 0.0};
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += 256) {
    s.sur += part[i].sur;
    s.kl += part[i].kl;
    s.clipped += part[i].clipped;
  }
  s.sur = block_sum(s.sur, red);
  s.kl = block_sum(s.kl, red);
  s.clipped = block_sum(s.clipped, red);
  if (threadIdx.x == 0) policy_stats(stats, s, kl_coef);
}

// Everything in one block: at most kSmallPieces pieces and kSmallSeqs sequences.
__global__ void __launch_bounds__(1024) policy_small_kernel(PolicyArgs a, PolicyConst k, unsigned* err) {
  __shared__ double red[32], inv[kSmallSeqs], scale_s;
  __shared__ Pair2 whole[kSmallSeqs], head[kSmallPieces], tail[kSmallPieces];
  grid_dependency_wait();
  const Seqs q = seqs_of(a);
  const SeqSums sums = {whole, head, tail};
  int c0, c1;
  my_pieces(pieces_of(q.N), &c0, &c1);
  double t = threadIdx.x == 0 ? 1.0 : 0.0;
  if (a.reduction == ARCHEAD_REDUCE_SEQUENCE) {
    if (a.w) sums_pieces<false>(q, nullptr, nullptr, a.w, c0, c1, sums);
    __syncthreads();
    t = 0.0;
    for (int s0 = 0; s0 < q.B; s0 += 128) {
      const int s = s0 + (threadIdx.x >> 3);
      const double v = policy_seq_inv(a, sums, s < q.B ? s : q.B - 1, threadIdx.x & 7, 8);
      if (s < q.B && (threadIdx.x & 7) == 0) {
        inv[s] = v;
        t += v > 0.0;
      }
    }
  } else if (a.reduction == ARCHEAD_REDUCE_TOKEN) {
    t = weight_share(a, threadIdx.x, 1024);
  }
  t = block_sum(t, red);
  if (threadIdx.x == 0) scale_s = t > 0.0 ? 1.0 / t : 0.0;
  __syncthreads();
  PolicySums s = {0.0, 0.0, 0.0};
  policy_pieces(a, k, c0, c1, scale_s, inv, s);
  check_seqs(q, threadIdx.x, 1024, err);
  s.sur = block_sum(s.sur, red);
  s.kl = block_sum(s.kl, red);
  s.clipped = block_sum(s.clipped, red);
  if (threadIdx.x == 0) policy_stats(a.stats, s, a.kl_coef);
}

PolicyConst policy_const(const PolicyArgs& a) {
  const double hi = log1p(a.clip_high), lo = log1p(-a.clip_low);
  return {hi, lo, (float)hi, (float)lo, (float)(1.0 + a.clip_high), (float)(1.0 - a.clip_low), (float)a.kl_coef};
}

int64_t piece_count(int64_t N) { return (N + kPiece - 1) / kPiece; }
int capped(int64_t blocks) { return (int)(blocks < 1 ? 1 : (blocks > kMaxBlocks ? kMaxBlocks : blocks)); }

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
bool small_tokens(int64_t N, int64_t B) { return piece_count(N) <= kSmallPieces && B <= kSmallSeqs; }

// A launch that may start while the previous kernel of the stream runs (its kernel waits for
// it before reading its results).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), int64_t grid, int threads, size_t smem, cudaStream_t st,
                         A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// ---- preference loss --------------------------------------------------------------------
// A sequence's slope dL/df over its pairs, in fixed point: signed 64-bit limbs, limb k of weight
// 2^(32 k - 192), so sums up to 2^31 pairs keep every bit from 2^-192 to 2^127 (of the unit that the host
// chooses, about the largest slope of an ordinary pair: slopes of decided pairs fade as e^-m, and
// their FP32 gradients keep their precision down to the smallest) and integer adds make the
// result independent of their order.  A slope that is not finite, or 2^127 units or more, counts
// in one more word and makes the sequence's slope NaN.
constexpr int kLimbs = 10, kSlopeWords = kLimbs + 1;

__device__ __forceinline__ double pow2_double(int e) { return __longlong_as_double((long long)(1023 + e) << 52); }

__device__ __forceinline__ void slope_add(unsigned long long* acc, double v) {
  if (!(fabs(v) < 1.7014118346046923e38)) {
    atomicAdd(acc + kLimbs, 1ull);
    return;
  }
  const int e = ((__double2hiint(v) >> 20) & 0x7ff) - 1023;
  if (e < -192) return;
  const int k = (e + 192) >> 5;  // the limb of the leading bit; the 53 bits reach into two more
  v *= pow2_double(192 - 32 * k);  // exact, as are the steps below: powers of two and the fraction's bits
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const long long d = (long long)v;  // toward zero
    if (d && k >= j) atomicAdd(acc + (k - j), (unsigned long long)d);
    v = (v - (double)d) * 4294967296.0;
  }
}

__device__ __forceinline__ double slope_value(const unsigned long long* acc) {
  if (acc[kLimbs]) return __longlong_as_double(0x7ff8000000000000ll);
  double v = 0.0;
#pragma unroll
  for (int k = 0; k < kLimbs; ++k) v = fma((double)(long long)acc[k], pow2_double(32 * k - 192), v);
  return v;
}

struct PrefConst {
  double beta, smoothing, margin, unit;  // slopes are counted in units of 1 / `unit`
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
    // (without smoothing an infinite margin costs nothing)
    *loss = l + (m >= 0 ? (k.smoothing > 0.0 ? k.smoothing * m : 0.0) : -(1.0 - k.smoothing) * m);
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

__device__ __forceinline__ Seqs seqs_of(const PreferenceArgs& a) { return {a.cu, (int)a.N, (int)a.B}; }

// Pair p by 16 lanes (eight per sequence; all lanes of a warp call it): its loss and rewards, its
// slope into both sequences' accumulators.  Its loss comes back in the first of the 16 lanes.
__device__ __forceinline__ double pair_step(const PreferenceArgs& a, const PrefConst& k, const SeqSums& q,
                                            int64_t p, unsigned long long* acc, unsigned* err) {
  const int lane = threadIdx.x & 31, half = (lane >> 3) & 1;
  const bool live = p < a.P;
  const int mine = live ? __ldg(a.pairs + 2 * p + half) : 0;
  const bool ok = mine >= 0 && mine < a.B;
  const Seqs sq = seqs_of(a);
  Pair2 t = {0.0, 0.0};
  // (the sums' shuffles need every lane; without sequences there is nothing to read)
  if (a.B > 0) t = seq_total(q, sq, ok ? mine : 0, lane & 7, 8);
  const double f = ok ? score_of(t, a.average) : __longlong_as_double(0x7ff8000000000000ll);
  const double fb = __shfl_xor_sync(0xffffffffu, f, 8);
  const int ib = __shfl_xor_sync(0xffffffffu, mine, 8);
  const bool okb = __shfl_xor_sync(0xffffffffu, (int)ok, 8);
  if (!live || (lane & 15) != 0) return 0.0;
  double loss = __longlong_as_double(0x7ff8000000000000ll), slope;
  if (ok && okb) {
    pref_pair(f - fb, k, &loss, &slope);
    slope_add(acc + (int64_t)mine * kSlopeWords, slope * k.unit);
    slope_add(acc + (int64_t)ib * kSlopeWords, -slope * k.unit);
  } else {
    atomicOr(err, kErrSegment);
  }
  a.pair_loss[p] = (float)loss;
  a.rewards[2 * p] = (float)(ok && okb ? k.beta * f : loss);
  a.rewards[2 * p + 1] = (float)(ok && okb ? k.beta * fb : loss);
  return loss;
}

// dnll[t] = -w [/ sum w] slope(sequence) / P for pieces [c, c1).
__device__ __forceinline__ void pref_pieces(const PreferenceArgs& a, const PrefConst& k, const SeqSums& q,
                                            const unsigned long long* acc, int c, int c1) {
  const Seqs sq = seqs_of(a);
  const int lane = threadIdx.x & 31;
  if (c >= c1) return;
  const double per_pair = a.P ? 1.0 / (k.unit * (double)a.P) : 0.0;
  const bool vec = aligned16(a.w, a.dnll);
  double coef = 0.0;  // of the window's sequence
  auto window = [&](int s) { coef = -slope_value(acc + (int64_t)s * kSlopeWords) * per_pair; };
  Walker<decltype(window)> walk(sq, c * kPiece, window);
  // With `average`: the last sequence's weight.  A long one comes back in every piece of the warp; added
  // up from its pieces each time, 2^31 tokens of one sequence took 100 s a call.
  int weighed = -1;
  double weight = 0.0;
  for (; c < c1; ++c) {
    const int t0 = c * kPiece, t1 = sq.N - t0 < kPiece ? sq.N : t0 + kPiece;
    float w[kPer], g[kPer] = {};
    load_piece(a.w, t0, t1, vec, a.w ? 0.f : 1.f, w);
    walk.piece(t0, t1, [&](int j, int s, int lo, int hi, int, int) {
      double f = __shfl_sync(0xffffffffu, coef, j);
      if (a.average) {
        if (s != weighed) {
          weight = seq_total(q, sq, s, lane, 32).w;
          weighed = s;
        }
        f = weight > 0.0 ? f / weight : 0.0;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const bool in = (unsigned)(token_at(t0, i) - lo) < (unsigned)(hi - lo);
        if (in && w[i] != 0.f) g[i] = (float)(f * (double)w[i]);
      }
    }, [&](int s, int lo, int hi, int b0, int b1, bool mine) {
      double own = coef;
      if (a.average) {
        const double t = mine && b1 > b0 ? q.whole[s + lane].w : 0.0;
        own = t > 0.0 ? own / t : 0.0;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int t = token_at(t0, i);
        const double f = __shfl_sync(0xffffffffu, own, lane_of(b1, t));
        const bool in = (unsigned)(t - lo) < (unsigned)(hi - lo);
        if (in && w[i] != 0.f) g[i] = (float)(f * (double)w[i]);
      }
    });
    store_piece(a.dnll, t0, t1, vec, g);
  }
}

// With few sequences (kFew) many pairs add to one slope: a block's are added in shared memory first
// (12000 pairs of 2 sequences: a call 41 -> 22 us).
constexpr int kLocalSeqs = 256;
template <bool kFew>
__global__ void __launch_bounds__(256) pref_pair_kernel(PreferenceArgs a, PrefConst k, SeqSums q,
                                                        unsigned long long* acc, double* part,
                                                        unsigned* err) {
  allow_dependent_launch();
  __shared__ double red[8];
  __shared__ unsigned long long local[kFew ? kLocalSeqs * kSlopeWords : 1];
  const int words = kFew ? (int)a.B * kSlopeWords : 0;
  for (int i = threadIdx.x; i < words; i += 256) local[i] = 0ull;
  if (kFew) __syncthreads();
  grid_dependency_wait();
  double sum = 0.0;
  for (int64_t p0 = blockIdx.x * 16ll; p0 < a.P; p0 += gridDim.x * 16ll)
    sum += pair_step(a, k, q, p0 + (threadIdx.x >> 4), kFew ? local : acc, err);
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
  for (int i = threadIdx.x; i < words; i += 256)
    if (local[i]) atomicAdd(acc + i, local[i]);
}

__device__ __forceinline__ float pref_mean(const PreferenceArgs& a, double sum) {
  return a.P ? (float)(sum / (double)a.P) : 0.f;
}

// Block 0 also adds the losses.
__global__ void __launch_bounds__(256, 4) pref_token_kernel(PreferenceArgs a, PrefConst k, SeqSums q,
                                                         const unsigned long long* acc,
                                                         const double* part, int npart) {
  grid_dependency_wait();
  __shared__ double red[8];
  if (blockIdx.x == 0) {
    double s = 0.0;
    for (int i = threadIdx.x; i < npart; i += 256) s += part[i];
    s = block_sum(s, red);
    if (threadIdx.x == 0) a.loss[0] = pref_mean(a, s);
  }
  int c0, c1;
  my_pieces(pieces_of(a.N), &c0, &c1);
  pref_pieces(a, k, q, acc, c0, c1);
}

// Everything in one block: at most kSmallPieces pieces, kSmallSeqs sequences, kSmallPairs pairs.
// Dynamic shared memory: B accumulators.
__global__ void __launch_bounds__(1024) pref_small_kernel(PreferenceArgs a, PrefConst k, unsigned* err) {
  extern __shared__ unsigned long long acc[];
  __shared__ double red[32];
  __shared__ Pair2 whole[kSmallSeqs], head[kSmallPieces], tail[kSmallPieces];
  grid_dependency_wait();
  const Seqs sq = seqs_of(a);
  const SeqSums sums = {whole, head, tail};
  int c0, c1;
  my_pieces(pieces_of(sq.N), &c0, &c1);
  sums_pieces<true>(sq, a.nll, a.nll_ref, a.w, c0, c1, sums);
  for (int i = threadIdx.x; i < sq.B * kSlopeWords; i += 1024) acc[i] = 0ull;
  __syncthreads();
  double sum = 0.0;
  for (int64_t p0 = 0; p0 < a.P; p0 += 64) sum += pair_step(a, k, sums, p0 + (threadIdx.x >> 4), acc, err);
  __syncthreads();
  pref_pieces(a, k, sums, acc, c0, c1);
  check_seqs(sq, threadIdx.x, 1024, err);
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) a.loss[0] = pref_mean(a, sum);
}

PrefConst pref_const(const PreferenceArgs& a) {
  PrefConst k = {a.beta, a.smoothing, a.margin, 1.0, a.kind};
  // the largest slope of an ordinary pair: beta, or 1 / beta for ipo
  k.unit = ldexp(1.0, -ilogb(a.kind == ARCHEAD_PREF_IPO ? fmax(1.0, 1.0 / a.beta) : a.beta));
  return k;
}

bool pref_small(const PreferenceArgs& a) { return small_tokens(a.N, a.B) && a.P <= kSmallPairs; }

}  // namespace

size_t policy_scratch_bytes(const PolicyArgs& a) {
  if (small_tokens(a.N, a.B)) return 0;
  size_t b = up256(kMaxBlocks * sizeof(PolicySums)) + up256(kMaxBlocks * 8);
  if (a.reduction == ARCHEAD_REDUCE_SEQUENCE)
    b += up256((size_t)a.B * 8) + (a.w ? seq_sum_bytes(a.N, a.B) : 0);
  return b;
}

cudaError_t launch_policy_loss(const PolicyArgs& a, void* scratch, unsigned* err,
                               cudaStream_t st, int* launches) {
  const PolicyConst k = policy_const(a);
  if (small_tokens(a.N, a.B)) {
    ++*launches;
    return launch_after(policy_small_kernel, 1, 1024, 0, st, a, k, err);
  }
  char* b = static_cast<char*>(scratch);
  PolicySums* part = reinterpret_cast<PolicySums*>(b);
  b += up256(kMaxBlocks * sizeof(PolicySums));
  double* total = reinterpret_cast<double*>(b);
  b += up256(kMaxBlocks * 8);
  const int64_t pb = (piece_count(a.N) + 7) / 8;
  // blocks of the token kernels (three per SM: the tokens in flight take 80 registers)
  const int nb = capped(pb) < 148 * 3 ? capped(pb) : 148 * 3;
  int nt = 0;
  double* inv = nullptr;
  cudaError_t e = cudaSuccess;
  if (a.reduction == ARCHEAD_REDUCE_TOKEN) {
    nt = nb;
    policy_weight_kernel<<<nt, 256, 0, st>>>(a, total, err);
    ++*launches;
    e = cudaGetLastError();
  } else if (a.reduction == ARCHEAD_REDUCE_SEQUENCE) {
    inv = reinterpret_cast<double*>(b);
    b += up256((size_t)a.B * 8);
    SeqSums q = {};
    if (a.w) {
      q = carve_seq_sums(b, a.N, a.B);
      const Seqs sq = {a.cu, (int)a.N, (int)a.B};
      seq_sums_kernel<false><<<nb, 256, 0, st>>>(nullptr, nullptr, a.w, sq, q, nullptr, 0, err);
      ++*launches;
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    nt = capped((a.B + 31) / 32) < 256 ? capped((a.B + 31) / 32) : 256;
    e = launch_after(policy_seq_kernel, nt, 256, 0, st, a, q, inv, total, err);
    ++*launches;
  }
  if (e != cudaSuccess) return e;
  e = launch_after(policy_token_kernel, nb, 256, 0, st, a, k, inv, nt ? total : nullptr, nt, part, err);
  if (e != cudaSuccess) return e;
  *launches += 2;
  return launch_after(policy_final_kernel, 1, 256, 0, st, part, nb, a.kl_coef, a.stats);
}

size_t preference_scratch_bytes(const PreferenceArgs& a) {
  if (pref_small(a)) return 0;
  return up256(8 * kMaxBlocks) + up256((size_t)a.B * kSlopeWords * 8) + seq_sum_bytes(a.N, a.B);
}

cudaError_t launch_preference_loss(const PreferenceArgs& a, void* scratch, unsigned* err,
                                   cudaStream_t st, int* launches) {
  const PrefConst k = pref_const(a);
  if (pref_small(a)) {
    ++*launches;
    return launch_after(pref_small_kernel, 1, 1024, (size_t)a.B * kSlopeWords * 8, st, a, k, err);
  }
  char* b = static_cast<char*>(scratch);
  double* part = reinterpret_cast<double*>(b);
  b += up256(8 * kMaxBlocks);
  unsigned long long* acc = reinterpret_cast<unsigned long long*>(b);
  b += up256((size_t)a.B * kSlopeWords * 8);
  const SeqSums q = carve_seq_sums(b, a.N, a.B);
  const Seqs sq = {a.cu, (int)a.N, (int)a.B};
  const int pb = capped((piece_count(a.N) + 7) / 8);
  seq_sums_kernel<true><<<pb, 256, 0, st>>>(a.nll, a.nll_ref, a.w, sq, q, acc, a.B * kSlopeWords, err);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int np = capped((a.P + 15) / 16);
  e = launch_after(a.B <= kLocalSeqs ? pref_pair_kernel<true> : pref_pair_kernel<false>, np, 256, 0, st, a, k, q, acc, part, err);
  if (e != cudaSuccess) return e;
  e = launch_after(pref_token_kernel, pb, 256, 0, st, a, k, q, acc, part, np);
  *launches += 3;
  return e;
}

}  // namespace archead
