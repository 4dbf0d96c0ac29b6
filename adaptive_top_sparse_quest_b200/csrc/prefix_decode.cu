// Dense decode attention of a batch whose sequences share their first tokens
// (tw_prefix_decode):
//   out_b,hq = sum_{t < len_b} softmax_t(q_b,hq . k_b,t / sqrt(128)) v_b,t,
// tokens t < prefix_len being the same rows for every sequence.
//
// First form: one block per (sequence, KV head) walks all tokens of its
// sequence, a half-warp per token with the running maximum and sum of the
// softmax in registers, and folds its half-warps at the end.  The prefix is
// read once per sequence.
#include "tw_common.cuh"
#include "tw_kernels.h"

namespace tw {

constexpr int kPdThreads = 128;
constexpr int kPdHW = kPdThreads / 16;

template <int G>
__global__ void __launch_bounds__(kPdThreads)
k_prefix_decode(Layout L, const __half* __restrict__ q, int Hq, int P, const __half* __restrict__ K,
                const __half* __restrict__ V, __half* __restrict__ out, float* __restrict__ lse) {
  __shared__ float sm_m[kPdHW][G], sm_l[kPdHW][G], sm_acc[kPdHW][G][kHeadDim];
  const int tid = threadIdx.x, lane = tid & 31, hw = tid >> 4, l16 = tid & 15;
  const unsigned hmask = 0xFFFFu << (lane & 16);
  const int b = blockIdx.x / L.Hk, h = blockIdx.x % L.Hk;
  const int len = L.len(b);
  const float scale = 1.4426950408889634f * 0.08838834764831845f;   // log2(e) / sqrt(128)
  float qf[G][8], m[G], l[G], acc[G][8];
  for (int g = 0; g < G; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
    for (int j = 0; j < 8; ++j) {
      qf[g][j] = __half2float(q[((int64_t)b * Hq + h * G + g) * kHeadDim + 8 * l16 + j]) * scale;
      acc[g][j] = 0.f;
    }
  }
  for (int t = hw; t < len; t += kPdHW) {
    const int64_t row = L.row(t < P ? 0 : b, h, t);
    const __half* kr = K + row * kHeadDim + 8 * l16;
    const __half* vr = V + row * kHeadDim + 8 * l16;
    for (int g = 0; g < G; ++g) {
      float s = 0.f;
      for (int j = 0; j < 8; ++j) s = __fmaf_rn(qf[g][j], __half2float(kr[j]), s);
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(hmask, s, o, 16);
      const float mb = fmaxf(m[g], s), corr = exp2f(m[g] - mb), p = exp2f(s - mb);
      l[g] = l[g] * corr + p;
      for (int j = 0; j < 8; ++j) acc[g][j] = __fmaf_rn(p, __half2float(vr[j]), acc[g][j] * corr);
      m[g] = mb;
    }
  }
  for (int g = 0; g < G; ++g) {
    sm_m[hw][g] = m[g];
    sm_l[hw][g] = l[g];
    for (int j = 0; j < 8; ++j) sm_acc[hw][g][8 * l16 + j] = acc[g][j];
  }
  __syncthreads();
  for (int g = 0; g < G; ++g) {
    float M = -INFINITY, Ls = 0.f, A = 0.f;
    for (int w = 0; w < kPdHW; ++w) M = fmaxf(M, sm_m[w][g]);
    for (int w = 0; w < kPdHW; ++w) {
      const float f = sm_m[w][g] == -INFINITY ? 0.f : exp2f(sm_m[w][g] - M);
      Ls += sm_l[w][g] * f;
      A += sm_acc[w][g][tid] * f;
    }
    const int64_t bh = (int64_t)b * Hq + h * G + g;
    out[bh * kHeadDim + tid] = __float2half_rn(Ls > 0.f ? A / Ls : 0.f);
    if (lse && tid == 0)
      lse[bh] = Ls > 0.f ? (M + log2f(Ls)) * 0.6931471805599453f : -INFINITY;
  }
}

size_t prefix_decode_ws_bytes(int, int, int, int) { return 256; }

cudaError_t launch_prefix_decode(const Layout& L, const __half* q, int Hq, int prefix_len,
                                 const __half* K, const __half* V, __half* out, float* lse, void*,
                                 cudaStream_t st) {
  const dim3 grid(L.B * L.Hk), block(kPdThreads);
  switch (Hq / L.Hk) {
#define TW_PD(NN) \
  case NN:        \
    return launch_k(k_prefix_decode<NN>, grid, block, 0, st, false, L, q, Hq, prefix_len, K, V, out, lse);
    TW_PD(1) TW_PD(2) TW_PD(4) TW_PD(8)
#undef TW_PD
  }
  return cudaErrorInvalidValue;
}

}  // namespace tw
