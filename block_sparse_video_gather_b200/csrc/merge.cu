// merge.cu -- untile fused with the merge of the fine stage's output and an
// attention over other keys (the cached past of a video made chunk by chunk).
//
// Two attentions of one query over disjoint key sets, with lse l1 and l2, are
// the attention over the union: weights exp(l_i) / (exp(l1) + exp(l2)), lse =
// log(exp(l1) + exp(l2)).  With m = max(l1, l2), w_i = exp(l_i - m) is in
// [0, 1] and the larger is 1, so the sum is in [1, 2]; a side of -inf gets
// weight 0 and its o, which may be anything, is not read into the sum.  A NaN in
// either makes the row NaN.
// Bound: HBM (two 16-bit reads and one write a channel, 12 bytes a row).  One
// CTA per (64 tiled rows, b, h), heads the fast index, so that CTAs that run
// together touch the same tokens' rows; a thread owns one 16-byte chunk of 4
// rows, all loaded at once.  A row's weights are made by one lane for its 16
// threads: with two exponentials, a logarithm and a quotient in every thread
// the arithmetic took longer than the traffic (64 us for the 306 MB of a
// (21, 30, 52) grid and 12 heads; now 52.7 alone, 54.7 with the next call behind
// it, 5.6 to 5.8 TB/s).
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

constexpr int kMergeRows = 64;
constexpr int kMergeIters = kMergeRows / (kTileThreads / kRowChunks);  // rows of a thread

template <int BS, bool F16>
__global__ void __launch_bounds__(kTileThreads) untile_merge_kernel(Geo g, int H, int BH,
                                                                    const uint4* __restrict__ ot,
                                                                    const float* __restrict__ lse_t,
                                                                    const uint4* past, const float* lse_past,
                                                                    uint4* o, float* lse) {
  constexpr int kParts = BS / kMergeRows;
  const int at = blockIdx.x / BH, bh = blockIdx.x - at * BH;
  const int blk = at / kParts, first = (at - blk * kParts) * kMergeRows;
  const int b = bh / H, h = bh - b * H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = lane & (kRowChunks - 1), upper = lane >> 4;
  const long long srow = static_cast<long long>(bh) * g.Sp + static_cast<long long>(blk) * BS + first;

  // lane 2 i + u looks after row 2 warp + u of the i-th 16: where it goes and its weights
  long long dst = -1;
  float l1 = 0.0f, l2 = 0.0f;
  if (lane < 2 * kMergeIters) {
    const int row = 2 * warp + (lane & 1) + 16 * (lane >> 1);
    const long long s = token_of_slot(g, block_origin(g, blk), first + row);
    if (s >= 0) {
      dst = (static_cast<long long>(b) * g.S + s) * H + h;
      l1 = __ldg(lse_t + srow + row);
      l2 = lse_past[dst];
    }
  }
  uint4 x[kMergeIters], y[kMergeIters];
  long long to[kMergeIters];
#pragma unroll
  for (int i = 0; i < kMergeIters; ++i) {
    to[i] = __shfl_sync(0xffffffffu, dst, 2 * i + upper);
    x[i] = y[i] = make_uint4(0, 0, 0, 0);
    if (to[i] >= 0) {
      x[i] = __ldcs(ot + (srow + 2 * warp + upper + 16 * i) * kRowChunks + chunk);
      y[i] = __ldcs(past + to[i] * kRowChunks + chunk);
    }
  }
  const float m = fmaxf(l1, l2);
  const bool none = l1 == -INFINITY && l2 == -INFINITY;  // by each: fmaxf drops a NaN
  const float w1 = l1 == -INFINITY ? 0.0f : expf(l1 - m);
  const float w2 = l2 == -INFINITY ? 0.0f : expf(l2 - m);
  const float sum = w1 + w2;
  const float s1 = none ? 0.0f : w1 / sum, s2 = none ? 0.0f : w2 / sum;
  if (lse != nullptr && dst >= 0) lse[dst] = none ? -INFINITY : m + logf(sum);
#pragma unroll
  for (int i = 0; i < kMergeIters; ++i) {
    const float a = __shfl_sync(0xffffffffu, s1, 2 * i + upper), c = __shfl_sync(0xffffffffu, s2, 2 * i + upper);
    if (to[i] < 0) continue;
    const uint32_t xw[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    const uint32_t yw[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = pair_of<F16>(xw[j]), q = pair_of<F16>(yw[j]);
      float lo = 0.0f, hi = 0.0f;
      if (a != 0.0f) {
        lo = a * p.x;
        hi = a * p.y;
      }
      if (c != 0.0f) {
        lo = __fmaf_rn(c, q.x, lo);
        hi = __fmaf_rn(c, q.y, hi);
      }
      r[j] = pack_half2<F16>(lo, hi);
    }
    __stcs(o + to[i] * kRowChunks + chunk, make_uint4(r[0], r[1], r[2], r[3]));
  }
}

}  // namespace

cudaError_t launch_untile_merge(const Geo& g, int B, int H, const uint16_t* ot, const float* lse_t,
                                const uint16_t* past, const float* lse_past, uint16_t* o, float* lse, bool f16,
                                cudaStream_t stream) {
  const long long grid = static_cast<long long>(g.NB) * (g.bs / kMergeRows) * B * H;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const uint4* oi = reinterpret_cast<const uint4*>(ot);
  const uint4* pi = reinterpret_cast<const uint4*>(past);
  uint4* oo = reinterpret_cast<uint4*>(o);
  auto kern = g.bs == 256 ? (f16 ? untile_merge_kernel<256, true> : untile_merge_kernel<256, false>)
                          : (f16 ? untile_merge_kernel<64, true> : untile_merge_kernel<64, false>);
  kern<<<static_cast<unsigned>(grid), kTileThreads, 0, stream>>>(g, H, B * H, oi, lse_t, pi, lse_past, oo, lse);
  return cudaGetLastError();
}

}  // namespace vsa
