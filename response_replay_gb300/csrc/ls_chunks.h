// ls_chunks.h -- the chunks of a row that is streamed through shared memory.  Included by host and
// device code.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define LS_CHUNK_FN __host__ __device__ __forceinline__
#else
#define LS_CHUNK_FN inline
#endif

// Bytes of chunk k of a row of n groups of kGroup bytes, kPer groups a chunk (k kPer < n).  Counted
// in groups: a row of 2^30 values passes 2^31 bytes.
template <int kGroup, int kPer>
LS_CHUNK_FN uint32_t ls_chunk_bytes(int32_t n, int32_t k) {
  const int32_t left = n - k * kPer;
  return (uint32_t)(left < kPer ? left : kPer) * kGroup;
}
