// Rank products t = H' [Q8(B_c) | Q8(B_w)]^T of the tcgen05 path on warp MMAs, from the FP16 image
// of H' = H 2^-e_n into the image's rank blocks (tc_image_offset).
//
//   t[n, j] = sum_k s[j, k] sum_{d in group k} h'[n, d] q[j, d]
//
// q is INT8, exact in FP16; a group's products accumulate in FP32 from 0 and are added with the
// group's scale, so t has FP32 accuracy like the CUDA-core kernel's.  One block per 32 tokens x 32
// ranks, a warp per 16 x 16 of them; 128 columns of both operands per stage of a cp.async ring.  The
// operands are small (H once per 32 ranks), so the ring's latency bounds it.
#include "grad_common.cuh"

namespace archead {
namespace {

constexpr int kStages = 3;
constexpr int kHBytes = 32 * 256, kQRow = 144, kQBytes = 32 * kQRow;  // a stage: 32 x 128 FP16, 32 x 128 INT8

struct LowrankParams {
  archead_head h;
  __half* img;
  int64_t n, nkbt;
  int nt;
  unsigned* err;
};

__global__ void __launch_bounds__(128) lowrank_mma_kernel(const LowrankParams p) {
  allow_dependent_launch();
  __shared__ __align__(128) unsigned char sm[kStages * (kHBytes + kQBytes)];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gr = lane >> 2, q = lane & 3;
  const int RR = p.h.r_c + p.h.r_r;
  const int nkb = (int)(p.h.D >> 7);
  const int64_t G = p.h.D / p.h.g;
  const int64_t n0 = blockIdx.x * 32ll;  // (nt is a multiple of 32 here)
  const int j0 = blockIdx.y * 32;
  const int64_t tt = n0 / p.nt;
  const int nn0 = (int)(n0 - tt * p.nt);
  const char* himg = reinterpret_cast<const char*>(p.img) + tt * p.nkbt * p.nt * 256 + nn0 * 128;
  auto row_of = [&](int j) { return j < p.h.r_c ? p.h.Bc + j * p.h.D : p.h.Bw + (j - p.h.r_c) * p.h.D; };
  auto load = [&](int kb) {  // block kb into its stage; rows past the ranks are zeros
    unsigned char* H = sm + (kb % kStages) * (kHBytes + kQBytes);
    unsigned char* Q = H + kHBytes;
    if (kb < nkb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // two 64-column halves of 32 rows x 128 bytes, swizzle kept
        const int c = tid + 128 * i, half = c >> 8, o = (c & 255) * 16;
        cp_async16(H + half * 4096 + o, himg + ((int64_t)kb * 2 + half) * p.nt * 128 + o);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = tid + 128 * i, j = c >> 3, o = (c & 7) * 16;
        const bool in = j0 + j < RR;
        cp_async16_zfill(Q + j * kQRow + o, row_of(in ? j0 + j : 0) + kb * 128 + o, in ? 16 : 0);
      }
    }
    cp_async_commit();
  };
  grid_dependency_wait();
  for (int i = 0; i < kStages - 1; ++i) load(i);
  const int m0 = 16 * (warp & 1), c0 = 16 * (warp >> 1);  // this warp's tokens and ranks
  float t[2][4] = {}, acc[2][4];
  const int per = p.h.g >> 4;  // K steps of 16 per group
  int left = per;
  int64_t grp = 0;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[c][e] = 0.f;
  for (int kb = 0; kb < nkb; ++kb) {
    cp_async_wait<kStages - 2>();
    __syncthreads();  // stage kb has arrived, and the stage refilled next has been read
    load(kb + kStages - 1);
    const unsigned char* H = sm + (kb % kStages) * (kHBytes + kQBytes);
    const unsigned char* Q = H + kHBytes;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = m0 + (lane & 15), chunk = 2 * (k & 3) + (lane >> 4);
      const uint32_t at = tc::smem_u32(H + (k >> 2) * 4096 + r * 128 + (((chunk ^ (nn0 + r)) & 7) << 4));
      uint32_t a[4];
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                   : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                   : "r"(at));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const unsigned char* b = Q + (c0 + 8 * c + gr) * kQRow + 16 * k + 2 * q;
        const uint32_t x = *reinterpret_cast<const uint16_t*>(b) ^ 0x8080u;
        const uint32_t y = *reinterpret_cast<const uint16_t*>(b + 8) ^ 0x8080u;
        mma_f16_16816(acc[c], a, h2_bits(bytes_to_half2(x, 0x4140)), h2_bits(bytes_to_half2(y, 0x4140)));
      }
      if (--left == 0) {  // end of a group: its sums times its scales
        left = per;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = j0 + c0 + 8 * c + 2 * q + e;
            const float s = j >= RR ? 0.f : (j < p.h.r_c ? __ldg(p.h.sBc + j * G + grp) : __ldg(p.h.sBw + (j - p.h.r_c) * G + grp));
            t[c][e] = fmaf(acc[c][e], s, t[c][e]);
            t[c][2 + e] = fmaf(acc[c][2 + e], s, t[c][2 + e]);
            acc[c][e] = acc[c][2 + e] = 0.f;
          }
        ++grp;
      }
    }
  }
  bool bad = false;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = j0 + c0 + 8 * c + 2 * q + (e & 1);
      const int64_t n = n0 + m0 + gr + 8 * (e >> 1);
      if (j >= RR || n >= p.n) continue;
      const float v = t[c][e];
      const __half t1 = __float2half_rn(v);
      const __half t2 = __float2half_rn(v - __half2float(t1));
      bad |= !(fabsf(v) < 65504.f);
      const uint32_t w = (uint32_t)__half_as_ushort(t1) | ((uint32_t)__half_as_ushort(t2) << 16);
      *reinterpret_cast<uint2*>(p.img + tc_image_offset(tt, nkb + j / 32, p.nkbt, p.nt, (int64_t)(n - tt * p.nt),
                                                        4 * (j & 31))) = make_uint2(w, w);
    }
  if (bad) atomicOr(p.err, kErrRangeH);
}

}  // namespace

cudaError_t launch_lowrank_mma(const archead_head* head, const Shapes& s, const TcPlan& plan, __half* img,
                               unsigned* err, cudaStream_t st, int* launches) {
  const int RR = s.r_c + s.r_r;
  if (RR == 0) return cudaSuccess;
  const LowrankParams p = {*head, img, s.N, s.D / 128 + plan.nrb, plan.nt, err};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((s.N + 31) / 32), (unsigned)((RR + 31) / 32));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ++*launches;
  return cudaLaunchKernelEx(&cfg, lowrank_mma_kernel, p);
}

}  // namespace archead
