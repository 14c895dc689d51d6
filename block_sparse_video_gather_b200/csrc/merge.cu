// merge.cu -- untile fused with the merge of the fine stage's output and an
// attention over other keys (the cached past of a video made chunk by chunk).
//
// Two attentions of one query over disjoint key sets, with lse l1 and l2, are
// the attention over the union: weights exp(l_i) / (exp(l1) + exp(l2)), lse =
// log(exp(l1) + exp(l2)).  With m = max(l1, l2), w_i = exp(l_i - m) is in
// [0, 1] and the larger is 1, so the sum is in [1, 2]; a side of -inf gets
// weight 0 and its o, which may be anything, is not read into the sum.
// Bound: HBM (two 16-bit reads and one write a channel, 12 bytes a row).  One
// CTA per (b, h, block) as in the plain untile; a thread owns one 16-byte
// chunk of BS / 16 rows, all loaded before the first is used.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_kernels.h"
#include "common.cuh"
#include "items.cuh"

namespace vsa {

namespace {

using namespace items;

template <bool F16>
__device__ __forceinline__ float2 pair_of(uint32_t w) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(bf16_lo(w), bf16_hi(w));
}

template <int BS, bool F16>
__global__ void __launch_bounds__(kTileThreads) untile_merge_kernel(Geo g, int H, const uint4* __restrict__ ot,
                                                                    const float* __restrict__ lse_t,
                                                                    const uint4* past, const float* lse_past,
                                                                    uint4* o, float* lse) {
  const int blk = blockIdx.x;
  const int bh = blockIdx.y;
  const int b = bh / H, h = bh - b * H;
  const int chunk = threadIdx.x & (kRowChunks - 1);
  const int row0 = threadIdx.x >> 4;
  constexpr int kIters = BS / 16;
  constexpr int kBatch = kIters < 4 ? kIters : 4;  // rows in flight
  const long long srow = static_cast<long long>(bh) * g.Sp + static_cast<long long>(blk) * BS;
  const BlockOrigin org = block_origin(g, blk);
#pragma unroll 1
  for (int i0 = 0; i0 < kIters; i0 += kBatch) {
    uint4 a[kBatch], c[kBatch];
    float l1[kBatch], l2[kBatch];
    long long dst[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = row0 + 16 * (i0 + i);
      const long long s = token_of_slot(g, org, row);
      dst[i] = s < 0 ? -1 : (static_cast<long long>(b) * g.S + s) * H + h;
      a[i] = c[i] = make_uint4(0, 0, 0, 0);
      l1[i] = l2[i] = 0.0f;
      if (s >= 0) {
        a[i] = __ldcs(ot + (srow + row) * kRowChunks + chunk);
        c[i] = __ldcs(past + dst[i] * kRowChunks + chunk);
        l1[i] = __ldg(lse_t + srow + row);
        l2[i] = lse_past[dst[i]];
      }
    }
    __syncwarp();  // a row's 16 threads have read lse_past before one of them may overwrite it
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (dst[i] < 0) continue;
      const float m = fmaxf(l1[i], l2[i]);
      const bool none = m == -INFINITY;
      const float w1 = l1[i] == -INFINITY ? 0.0f : expf(l1[i] - m);
      const float w2 = l2[i] == -INFINITY ? 0.0f : expf(l2[i] - m);
      const float sum = w1 + w2;
      const float s1 = none ? 0.0f : w1 / sum, s2 = none ? 0.0f : w2 / sum;
      const uint32_t aw[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
      const uint32_t cw[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
      uint32_t r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = pair_of<F16>(aw[j]), y = pair_of<F16>(cw[j]);
        float lo = 0.0f, hi = 0.0f;
        if (w1 != 0.0f) {
          lo = s1 * x.x;
          hi = s1 * x.y;
        }
        if (w2 != 0.0f) {
          lo = __fmaf_rn(s2, y.x, lo);
          hi = __fmaf_rn(s2, y.y, hi);
        }
        r[j] = pack_half2<F16>(lo, hi);
      }
      __stcs(o + dst[i] * kRowChunks + chunk, make_uint4(r[0], r[1], r[2], r[3]));
      if (lse != nullptr && chunk == 0) lse[dst[i]] = none ? -INFINITY : m + logf(sum);
    }
  }
}

}  // namespace

cudaError_t launch_untile_merge(const Geo& g, int B, int H, const uint16_t* ot, const float* lse_t,
                                const uint16_t* past, const float* lse_past, uint16_t* o, float* lse, bool f16,
                                cudaStream_t stream) {
  dim3 grid(g.NB, B * H);
  const uint4* oi = reinterpret_cast<const uint4*>(ot);
  const uint4* pi = reinterpret_cast<const uint4*>(past);
  uint4* oo = reinterpret_cast<uint4*>(o);
  auto kern = g.bs == 256 ? (f16 ? untile_merge_kernel<256, true> : untile_merge_kernel<256, false>)
                          : (f16 ? untile_merge_kernel<64, true> : untile_merge_kernel<64, false>);
  kern<<<grid, kTileThreads, 0, stream>>>(g, H, oi, lse_t, pi, lse_past, oo, lse);
  return cudaGetLastError();
}

}  // namespace vsa
