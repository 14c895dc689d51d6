// cache_kernels.h -- internal launch entry points of the 4-bit key/value cache
// and of the merge with the fine stage (not public ABI).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "cache.cuh"
#include "common.cuh"

namespace vsa {

// A kernel's shared-memory limit, raised on its first launch on each device (the
// attribute call costs as much as a short launch).
class SmemAllowed {
 public:
  cudaError_t ensure(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<unsigned long long> done_{0};
};

// cache.cu
struct CacheTablesArgs {
  const int32_t *kv_len, *new_len;
  int R, log_page;
  const int32_t* free_pages;
  int n_free;
  const int32_t* free_start;
  int32_t* table;
  int max_pages;
  int32_t *kv_len_out, *cu, *slots;
  int max_tokens;
  int32_t* free_next;
  unsigned int* status;
};
cudaError_t launch_cache_tables(const CacheTablesArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_release(const uint8_t* drop, int R, int log_page, int32_t* kv_len, const int32_t* table,
                                 int max_pages, int32_t* free_pages, int n_free, int32_t* free_start,
                                 unsigned int* status, cudaStream_t stream);
cudaError_t launch_cache_append(bool f16, const uint16_t* k, const uint16_t* v, long long k_stride,
                                long long v_stride, const int32_t* slots, int T, int Hkv, uint8_t* pages,
                                int num_pages, int log_page, unsigned int* status, cudaStream_t stream);
cudaError_t launch_cache_read(bool f16, const int32_t* slots, int T, int Hkv, const uint8_t* pages, int num_pages,
                              int log_page, uint16_t* k, uint16_t* v, unsigned int* status, cudaStream_t stream);

// cache_attn.cu
size_t cache_attn_workspace_bytes(int Hq, int Hkv, int max_q);
cudaError_t launch_cache_attn(const cache::AttnArgs& a, bool f16, int max_q, int num_sms, cudaStream_t stream);

// cache_attn_small.cu: requests of more than `over` and at most `upto` rows (new tokens x query heads of a key
// head); `rows`: the largest number expected, which selects the row tile.
size_t cache_attn_small_workspace(int num_workers);
cudaError_t launch_cache_attn_small(const cache::AttnArgs& a, int over, int upto, bool f16, int rows, int num_sms,
                                    cudaStream_t stream);

// cache_attn_chunk.cu: requests of more than `over` rows.
size_t cache_attn_chunk_workspace(int num_workers);
cudaError_t launch_cache_attn_chunk(const cache::AttnArgs& a, int over, bool f16, int num_workers,
                                    cudaStream_t stream);

// merge.cu
cudaError_t launch_untile_merge(const Geo& g, int B, int H, const uint16_t* ot, const float* lse_t,
                                const uint16_t* past, const float* lse_past, uint16_t* o, float* lse, bool f16,
                                cudaStream_t stream);

}  // namespace vsa
