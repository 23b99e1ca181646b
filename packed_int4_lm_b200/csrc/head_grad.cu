// Gradient product through the packed head, dH = dY W (archead_logits_grad, and the second
// half of archead_nll_grad):
//
//   dH[n, d] = s_n ( sum_v dY[n, v] S_v c[v, d / g] q[v, d]  +  sum_j u[n, j] b[j, d] ),
//   u[n, j]  = sum_v dY[n, v] a[v, j],
//
// a = [Q8(A_c) | Q8(A_w)], b = [Q8(B_c) ; Q8(B_w)], s_n a factor per token.  The first form:
// FP32 on the CUDA cores, one block per 32 tokens x 128 columns.
#include "archead_internal.cuh"

namespace archead {
namespace {

struct GradParams {
  const float* dY;
  archead_head h;
  int64_t n;
  const float* rowscale;
  float* u;  // n x (r_c + r_r)
  __nv_bfloat16* dH;
};

__device__ __forceinline__ float weight_at(const archead_head& h, int64_t v, int64_t d) {
  if (h.format == ARCHEAD_FMT_ROW8)
    return (float)reinterpret_cast<const int8_t*>(h.r_nib)[v * h.D + d] * h.row_scale[v];
  const int within = (int)(d & 127), w = within >> 5, i = (within & 31) >> 3, i8 = within & 7;
  const uint32_t word = reinterpret_cast<const uint32_t*>(
      h.r_nib + nib_chunk_offset(v, d >> 7, h.D >> 7, i))[w];
  const int pos = (i8 & 1) ? 4 + (i8 >> 1) : (i8 >> 1);
  const int q = (int)((word >> (4 * pos)) & 15u);
  return (float)((q >= 8 ? q - 16 : q) * (int)h.r_code[v * (h.D / h.g) + d / h.g]) *
         bf16_bits_to_float(h.r_super[v]);
}

__global__ void __launch_bounds__(256) rank_product_kernel(const GradParams p) {
  const int RR = p.h.r_c + p.h.r_r, j = blockIdx.y;
  const int64_t n = blockIdx.x;
  float a = 0.f;
  for (int64_t v = threadIdx.x; v < p.h.V; v += 256) {
    const float e = j < p.h.r_c ? (float)p.h.Ac[v * p.h.r_c + j] * p.h.sAc[v]
                                : (float)p.h.Aw[v * p.h.r_r + (j - p.h.r_c)] * p.h.sAw[v];
    a = fmaf(p.dY[n * p.h.V + v], e, a);
  }
  __shared__ float red[8];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) a += red[i];
    p.u[n * RR + j] = a;
  }
}

__global__ void __launch_bounds__(256) head_grad_kernel(const GradParams p) {
  __shared__ float Ws[32][128], Ys[32][33];
  const int d = threadIdx.x & 127, half = threadIdx.x >> 7;
  const int64_t d0 = (int64_t)blockIdx.y * 128, n0 = (int64_t)blockIdx.x * 32;
  float acc[16] = {};
  for (int64_t v0 = 0; v0 < p.h.V; v0 += 32) {
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * 32; i += 256) {
      const int64_t n = n0 + (i >> 5), v = v0 + (i & 31);
      Ys[i >> 5][i & 31] = n < p.n && v < p.h.V ? p.dY[n * p.h.V + v] : 0.f;
    }
    for (int i = half; i < 32; i += 2)
      Ws[i][d] = v0 + i < p.h.V ? weight_at(p.h, v0 + i, d0 + d) : 0.f;
    __syncthreads();
    for (int v = 0; v < 32; ++v)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[k] = fmaf(Ys[half * 16 + k][v], Ws[v][d], acc[k]);
  }
  const int RR = p.h.r_c + p.h.r_r;
  const int64_t G = p.h.D / p.h.g, col = d0 + d;
  for (int k = 0; k < 16; ++k) {
    const int64_t n = n0 + half * 16 + k;
    if (n >= p.n) break;
    float a = acc[k];
    for (int j = 0; j < RR; ++j) {
      const bool core = j < p.h.r_c;
      const int jj = core ? j : j - p.h.r_c;
      const float b = (float)(core ? p.h.Bc : p.h.Bw)[jj * p.h.D + col] *
                      (core ? p.h.sBc : p.h.sBw)[jj * G + col / p.h.g];
      a = fmaf(p.u[n * RR + j], b, a);
    }
    const float s = p.rowscale ? p.rowscale[n] : 1.f;
    p.dH[n * p.h.D + col] = __float2bfloat16(s == 0.f ? 0.f : a * s);
  }
}

__global__ void __launch_bounds__(256) softmax_grad_kernel(float* Y, const int32_t* targets,
                                                           const float* nll, const float* lse,
                                                           const float* dnll, int64_t V,
                                                           unsigned* err) {
  const int64_t n = blockIdx.x;
  const int64_t t = targets[n];
  const bool bad = t < 0 || t >= V;
  if (bad && dnll[n] != 0.f && threadIdx.x == 0) atomicOr(err, kErrTarget);
  const float l = bad ? __int_as_float(0x7fc00000) : lse[n];
  for (int64_t v = threadIdx.x; v < V; v += 256)
    Y[n * V + v] = v == t ? expm1f(-nll[n]) : expf(Y[n * V + v] - l);
}

}  // namespace

size_t head_grad_scratch_bytes(const archead_head* head, int64_t n) {
  return (size_t)n * (head->r_c + head->r_r) * 4;
}

cudaError_t launch_head_grad(const float* dY, const archead_head* head, int64_t n,
                             const float* rowscale, uint16_t* dH, void* scratch,
                             cudaStream_t st, int* launches) {
  const GradParams p = {dY, *head, n, rowscale, static_cast<float*>(scratch),
                        reinterpret_cast<__nv_bfloat16*>(dH)};
  if (head->r_c + head->r_r > 0) {
    rank_product_kernel<<<dim3((unsigned)n, head->r_c + head->r_r), 256, 0, st>>>(p);
    ++*launches;
  }
  head_grad_kernel<<<dim3((unsigned)((n + 31) / 32), (unsigned)(head->D / 128)), 256, 0, st>>>(p);
  ++*launches;
  return cudaGetLastError();
}

cudaError_t launch_softmax_grad(float* Y, const int32_t* targets, const float* nll,
                                const float* lse, const float* dnll, int64_t n, int64_t V,
                                unsigned* err, cudaStream_t st, int* launches) {
  softmax_grad_kernel<<<(unsigned)n, 256, 0, st>>>(Y, targets, nll, lse, dnll, V, err);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace archead
