// cache_attn.cu -- attention over the 4-bit key/value cache.
//
// One warp per (new token, query head): every lane holds 4 channels of q and of
// the output, a key costs one reduction over the warp, and the softmax runs
// online in fp32 (running maximum and sum, the output rescaled when the
// maximum grows).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "cache_kernels.h"

namespace vsa {

namespace {

using namespace cache;

template <bool F16>
__global__ void __launch_bounds__(256) cache_attn_rows_kernel(const __grid_constant__ AttnArgs a) {
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(a.T) * a.Hq) return;
  const int t = static_cast<int>(row / a.Hq), hq = static_cast<int>(row - static_cast<long long>(t) * a.Hq);
  if (row == 0)
    for (int i = lane; i < a.R; i += 32) load_request(a, i, true);  // reports what it has to cut
  // the request that holds token t
  int r = 0;
  Request req = load_request(a, 0, false);
  while (t >= req.q0 + req.n || t < req.q0) {
    if (++r == a.R) return;
    req = load_request(a, r, false);
  }
  const int h = hq / a.G, limit = visible(a, req, t - req.q0);
  const int ch = lane * 4;
  const uint2 qw = *reinterpret_cast<const uint2*>(a.q + t * a.q_stride + hq * 128 + ch);
  float q[4];
  if (F16) {
    const float2 x = f16x2_to_f32(qw.x), y = f16x2_to_f32(qw.y);
    q[0] = x.x, q[1] = x.y, q[2] = y.x, q[3] = y.y;
  } else {
    q[0] = bf16_lo(qw.x), q[1] = bf16_hi(qw.x), q[2] = bf16_lo(qw.y), q[3] = bf16_hi(qw.y);
  }
  float m = -INFINITY, l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < limit; ++j) {
    const int page = __ldg(a.table + static_cast<long long>(r) * a.max_pages + (j >> a.log_page));
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) atomicCAS(a.status, 0u, (unsigned)VSA_ERR_BAD_INDEX);
      continue;
    }
    const int p = j & 15;
    const uint8_t* rec = a.pages + record_of((page << a.log_page) + (j & ((1 << a.log_page) - 1)), h, a.Hkv, a.log_page);
    // two lanes share a word of 8 codes
    const uint32_t kc = reinterpret_cast<const uint32_t*>(rec + p * 64)[lane >> 1];
    const uint32_t vc = reinterpret_cast<const uint32_t*>(rec + kRecV + p * 64)[lane >> 1];
    const int g = lane >> 2;
    const float ks = f16x2_to_f32(from_e4m3x2(rec[kRecKS + p * 8 + g])).x;
    const float vs = f16x2_to_f32(from_e4m3x2(rec[kRecVS + g * 16 + (p & 3) * 4 + (p >> 2)])).x;
    uint32_t x[4], y[4];
    from_e2m1x8(kc, x);
    from_e2m1x8(vc, y);
    const bool odd = lane & 1;
    const float2 k0 = f16x2_to_f32(odd ? x[2] : x[0]), k1 = f16x2_to_f32(odd ? x[3] : x[1]);
    const float2 v0 = f16x2_to_f32(odd ? y[2] : y[0]), v1 = f16x2_to_f32(odd ? y[3] : y[1]);
    float s = (q[0] * k0.x + q[1] * k0.y + q[2] * k1.x + q[3] * k1.y) * ks;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s);
    const float alpha = m == -INFINITY ? 0.0f : ex2_approx(m - mn);
    const float pr = ex2_approx(s - (mn == -INFINITY ? 0.0f : mn));  // a NaN stays one
    m = mn;
    l = l * alpha + pr;
    acc[0] = acc[0] * alpha + pr * vs * v0.x;
    acc[1] = acc[1] * alpha + pr * vs * v0.y;
    acc[2] = acc[2] * alpha + pr * vs * v1.x;
    acc[3] = acc[3] * alpha + pr * vs * v1.y;
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  uint2 w;
  w.x = pack_half2<F16>(acc[0] * inv, acc[1] * inv);
  w.y = pack_half2<F16>(acc[2] * inv, acc[3] * inv);
  *reinterpret_cast<uint2*>(a.o + row * 128 + ch) = w;
  if (lane == 0) a.lse[row] = l != 0.0f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

size_t cache_attn_workspace_bytes(int, int, int) { return 16; }

cudaError_t launch_cache_attn(const cache::AttnArgs& a, bool f16, int, int, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.T) * a.Hq;
  if (rows == 0) return cudaSuccess;
  auto kern = f16 ? cache_attn_rows_kernel<true> : cache_attn_rows_kernel<false>;
  kern<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace vsa
