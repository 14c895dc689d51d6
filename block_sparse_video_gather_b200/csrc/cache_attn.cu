// cache_attn.cu -- attention over the 4-bit key/value cache: which kernel takes
// which request.
#include "cache_kernels.h"

namespace vsa {

namespace {

constexpr int kWorkers = 160;  // CTAs of a call at most: one per SM, B200 has 148

// Requests of up to this many rows (new tokens times query heads of a key head)
// run the kernel for few rows, others the 256-row tiles of the tensor cores.
constexpr int kFewRows = 48;

}  // namespace

size_t cache_attn_workspace_bytes(int Hq, int Hkv, int max_q) {
  const bool many = static_cast<long long>(max_q) * (Hq / Hkv) > kFewRows;
  return cache_attn_small_workspace(kWorkers) + (many ? cache_attn_chunk_workspace(kWorkers) : 0);
}

cudaError_t launch_cache_attn(const cache::AttnArgs& a, bool f16, int max_q, int num_sms, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const int workers = num_sms < kWorkers ? num_sms : kWorkers;
  const long long rows = static_cast<long long>(max_q) * a.G;
  if (rows <= kFewRows)
    return launch_cache_attn_small(a, 0, 0x7fffffff, f16, static_cast<int>(rows), workers, stream);
  cache::AttnArgs b = a;
  b.ws = static_cast<char*>(a.ws) + cache_attn_small_workspace(kWorkers);
  cudaError_t e = launch_cache_attn_chunk(b, kFewRows, f16, workers, stream);
  if (e != cudaSuccess) return e;
  return launch_cache_attn_small(a, 0, kFewRows, f16, kFewRows, workers, stream);
}

}  // namespace vsa
