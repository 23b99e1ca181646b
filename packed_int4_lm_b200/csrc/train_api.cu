// C ABI of the training operators (archead.h): the gradient of the per-token NLL and of the
// logits through the packed head, and the losses on per-token NLLs.  Argument checks,
// scratch and dispatch.
#include <math.h>

#include <algorithm>

#include "archead_internal.cuh"

using namespace archead;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Tokens per chunk of the gradients: about 2 GB of scratch for the FP16 image (and FP32 logits,
// where those go through memory) and the product's sums, at most 65536 (the kernels' grids), and
// chunks of about equal size, whole token tiles of the product where that allows.
constexpr int64_t kChunkBytes = 2ll << 30;

int64_t grad_chunk(int64_t N, int64_t V, int64_t D, int bytes) {
  const int64_t most = std::min<int64_t>(std::max<int64_t>(kChunkBytes / (V * bytes + 8 * D), 1), 65536);
  const int64_t even = (N + (N + most - 1) / most - 1) / ((N + most - 1) / most);
  return std::min(N, even >= 256 ? std::min((even + 255) / 256 * 256, most) : even);
}
// The last chunk is shorter and may be split otherwise.
size_t chunk_scratch(const archead_head* head, int64_t N, int64_t chunk) {
  const size_t whole = head_grad_scratch_bytes(head, chunk);
  return N % chunk ? std::max(whole, head_grad_scratch_bytes(head, N % chunk)) : whole;
}

// Runs `launch` with scratch of the given size; the common end of every entry point here.
template <typename F>
int with_scratch(size_t bytes, cudaStream_t st, F launch) {
  void* base;
  unsigned* err;
  int rc = take_scratch(bytes, st, &base, &err);
  if (rc) return rc;
  int launches = 0;
  rc = launch(static_cast<char*>(base), err, &launches);
  if (base) cudaFreeAsync(base, st);
  if (rc == ARCHEAD_OK) set_last_launches(launches);
  return rc;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? ARCHEAD_OK : ARCHEAD_ERR_CUDA; }

int check_tokens(const int32_t* cu, const float* const* f, int nf, int64_t N, int64_t B) {
  if (N < 0 || N > 0x7fffffffLL || B < 0 || B >= 0x7fffffffLL) return ARCHEAD_ERR_SHAPE;
  if (cu && !aligned(cu, 4)) return ARCHEAD_ERR_ALIGN;
  for (int i = 0; i < nf; ++i)
    if (f[i] && !aligned(f[i], 4)) return ARCHEAD_ERR_ALIGN;
  return ARCHEAD_OK;
}

}  // namespace

extern "C" {

int archead_nll_grad(const uint16_t* H, const archead_head* head, const int32_t* targets,
                     const float* nll, const float* lse, const float* dnll, uint16_t* dH,
                     int64_t N, int64_t V, int64_t D, int r_c, int r_r, int g, void* stream) {
  int rc = validate_head_args(head, N, V, D, r_c, r_r, g);
  if (rc) return rc;
  if (N == 0) {
    set_last_launches(0);
    return ARCHEAD_OK;
  }
  if (!H || !targets || !nll || !lse || !dnll || !dH) return ARCHEAD_ERR_NULLPTR;
  if (!aligned(H, 16) || !aligned(dH, 16) || !aligned(targets, 4) || !aligned(nll, 4) ||
      !aligned(lse, 4) || !aligned(dnll, 4))
    return ARCHEAD_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // The tcgen05 kernel writes the image itself; the others leave logits in memory.  A short last
  // chunk may run on another kernel than the ones before it.
  auto fused = [&](int64_t n) { return tc_image_fits(head, Shapes{n, V, D, r_c, r_r, g}); };
  const int64_t chunk = grad_chunk(N, V, D, fused(N) ? 2 : 6);
  const int64_t yrows = std::max(fused(chunk) ? 0 : chunk, N % chunk && !fused(N % chunk) ? N % chunk : 0);
  const size_t yoff = ((size_t)yrows * V * 4 + 255) / 256 * 256;
  return with_scratch(yoff + chunk_scratch(head, N, chunk), st,
                      [&](char* b, unsigned* err, int* launches) {
    float* Y = reinterpret_cast<float*>(b);
    for (int64_t n0 = 0; n0 < N; n0 += chunk) {
      const Shapes s = {std::min(chunk, N - n0), V, D, r_c, r_r, g};
      const HeadGrad a = {head, s.N, b + yoff, err, st, launches};
      const SoftmaxTokens t = {targets + n0, nll + n0, lse + n0, dnll + n0};
      int rc;
      if (fused(s.N)) {
        TcImageRun run;
        TcImage image = {};
        rc = tc_image_begin(H + n0 * D, head, s, head_grad_image_tile(s.N), st, launches, &run);
        if (rc) return rc;
        rc = cuda_status(grad_rows(a));
        if (!rc) rc = cuda_status(grad_tokens(a, t, &image));
        rc = tc_image_end(head, s, image, st, launches, run, rc);
        if (!rc) rc = cuda_status(grad_targets(a, t));
      } else {
        rc = archead_logits(H + n0 * D, head, Y, s.N, V, D, r_c, r_r, g, stream);
        if (rc) return rc;
        *launches += archead_last_launches();
        rc = cuda_status(grad_rows(a));
        if (!rc) rc = cuda_status(grad_image_softmax(a, Y, t));
      }
      if (!rc) rc = cuda_status(grad_product(a, dnll + n0, dH + n0 * D));
      if (rc) return rc;
    }
    return static_cast<int>(ARCHEAD_OK);
  });
}

int archead_logits_grad(const float* dY, const archead_head* head, uint16_t* dH, int64_t N,
                        int64_t V, int64_t D, int r_c, int r_r, int g, void* stream) {
  int rc = validate_head_args(head, N, V, D, r_c, r_r, g);
  if (rc) return rc;
  if (N == 0) {
    set_last_launches(0);
    return ARCHEAD_OK;
  }
  if (!dY || !dH) return ARCHEAD_ERR_NULLPTR;
  if (!aligned(dY, 4) || !aligned(dH, 16)) return ARCHEAD_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t chunk = grad_chunk(N, V, D, 2);
  return with_scratch(chunk_scratch(head, N, chunk), st,
                      [&](char* b, unsigned* err, int* launches) {
    for (int64_t n0 = 0; n0 < N; n0 += chunk) {
      const HeadGrad a = {head, std::min(chunk, N - n0), b, err, st, launches};
      cudaError_t e = grad_amax(a, dY + n0 * V);
      if (e == cudaSuccess) e = grad_rows(a);
      if (e == cudaSuccess) e = grad_image_dy(a, dY + n0 * V);
      if (e == cudaSuccess) e = grad_product(a, nullptr, dH + n0 * D);
      if (e != cudaSuccess) return cuda_status(e);
    }
    return static_cast<int>(ARCHEAD_OK);
  });
}

int archead_policy_loss(const float* nll, const float* nll_old, const float* nll_ref,
                        const float* advantages, const float* weights,
                        const int32_t* cu_seqlens, float* dnll, float* stats, int64_t N,
                        int64_t B, int adv_per_seq, double clip_low, double clip_high,
                        double kl_coef, int reduction, void* stream) {
  const float* f[] = {nll, nll_old, nll_ref, advantages, weights, dnll, stats};
  const int rc = check_tokens(cu_seqlens, f, 7, N, B);
  if (rc) return rc;
  if (reduction < ARCHEAD_REDUCE_TOKEN || reduction > ARCHEAD_REDUCE_SUM) return ARCHEAD_ERR_SHAPE;
  if (!(clip_low >= 0.0 && clip_low < 1.0) || !(clip_high >= 0.0) || !isfinite(clip_high) ||
      !isfinite(kl_coef))
    return ARCHEAD_ERR_SHAPE;
  if (!stats || ((adv_per_seq || reduction == ARCHEAD_REDUCE_SEQUENCE) && !cu_seqlens))
    return ARCHEAD_ERR_NULLPTR;
  if (N > 0 && (!nll || !nll_old || (!advantages && !(adv_per_seq && B == 0)) || !dnll))
    return ARCHEAD_ERR_NULLPTR;
  const PolicyArgs a = {nll, nll_old, nll_ref, advantages, weights, cu_seqlens, dnll, stats,
                        N, B, adv_per_seq != 0, reduction, clip_low, clip_high,
                        nll_ref ? kl_coef : 0.0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return with_scratch(policy_scratch_bytes(a), st, [&](char* b, unsigned* err, int* launches) {
    return cuda_status(launch_policy_loss(a, b, err, st, launches));
  });
}

int archead_preference_loss(const float* nll, const float* nll_ref, const float* weights,
                            const int32_t* cu_seqlens, const int32_t* pairs, float* dnll,
                            float* loss, float* pair_loss, float* rewards, int64_t N, int64_t B,
                            int64_t P, int kind, int average, double beta,
                            double label_smoothing, double margin, void* stream) {
  const float* f[] = {nll, nll_ref, weights, dnll, loss, pair_loss, rewards};
  const int rc = check_tokens(cu_seqlens, f, 7, N, B);
  if (rc) return rc;
  if (P < 0 || P > 0x7fffffffLL || kind < ARCHEAD_PREF_SIGMOID || kind > ARCHEAD_PREF_IPO)
    return ARCHEAD_ERR_SHAPE;
  if (!(beta > 0.0) || !isfinite(beta) || !isfinite(1.0 / beta) || !isfinite(margin) ||
      !(label_smoothing >= 0.0 && label_smoothing < 1.0) ||
      (kind != ARCHEAD_PREF_SIGMOID && label_smoothing != 0.0))
    return ARCHEAD_ERR_SHAPE;
  if (!cu_seqlens || !loss) return ARCHEAD_ERR_NULLPTR;
  if (N > 0 && (!nll || !dnll)) return ARCHEAD_ERR_NULLPTR;
  if (P > 0 && (!pairs || !pair_loss || !rewards)) return ARCHEAD_ERR_NULLPTR;
  if (pairs && !aligned(pairs, 4)) return ARCHEAD_ERR_ALIGN;
  const PreferenceArgs a = {nll, nll_ref, weights, cu_seqlens, pairs, dnll, loss, pair_loss,
                            rewards, N, B, P, kind, average != 0, beta, label_smoothing, margin};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return with_scratch(preference_scratch_bytes(a), st,
                      [&](char* b, unsigned* err, int* launches) {
    return cuda_status(launch_preference_loss(a, b, err, st, launches));
  });
}

}  // extern "C"
