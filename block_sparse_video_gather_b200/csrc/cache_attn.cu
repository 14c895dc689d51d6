// cache_attn.cu -- attention over the 4-bit key/value cache: which kernel takes
// which request.
#include "cache_kernels.h"

namespace vsa {

namespace {

constexpr int kWorkers = 160;  // CTAs of a call at most: one per SM, B200 has 148

// Requests of up to this many rows (new tokens times query heads of a key head)
// run the kernel for few rows, others the 256-row tiles of the tensor cores.
// Measured over 8000 cached tokens, us, few rows / tensor cores: 1 request x 12
// heads, 40 rows 30.3 / 32.6, 64 rows 34.1 / 32.7; 9 requests of up to 64 rows x
// 3 heads 38.7 / 57.0, 32 x 8 heads 200 / 210 (some of their requests have fewer
// rows, so that with a lower border both kernels run).
constexpr int kFewRows = 64;

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
  // A batch of one request that may have many rows needs no second kernel for requests with few.
  const int over = a.R == 1 ? 0 : kFewRows;
  cache::AttnArgs b = a;
  b.ws = static_cast<char*>(a.ws) + cache_attn_small_workspace(kWorkers);
  if (over != 0) b.fill = 0;  // the second kernel does it
  cudaError_t e = launch_cache_attn_chunk(b, over, f16, workers, stream);
  if (e != cudaSuccess || over == 0) return e;
  return launch_cache_attn_small(a, 0, kFewRows, f16, kFewRows, workers, stream);
}

}  // namespace vsa
