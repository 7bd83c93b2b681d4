// What the kernels over a paged key-value cache share (kv_cache.cu, kv8.cu): the checks of a call's list and of lengths.
#pragma once
#include "kernels.h"

namespace rpp {

namespace {

constexpr int kMoveThreads = 256;

__device__ __forceinline__ int used_pages(int len, int page_size) { return (len + page_size - 1) / page_size; }
__device__ __forceinline__ bool len_ok(int len, const KvDims& d) {
  return len >= 0 && static_cast<long long>(len) <= static_cast<long long>(d.max_pages) * d.page_size;
}

// The first words of a kernel that takes a list of slots: one reading of the error word for the
// whole CTA (other CTAs may set it at any time) and the list against the cache.  False if the CTA must
// quit: the word is set, or a slot lies outside [0, d.slots) or is given twice, or cu[i + 1] < cu[i]
// (recorded by one thread; every CTA of a launch comes to the same answer).  `seen`: (d.slots + 31) / 32
// words of shared memory, left holding the slots given; cu: [n + 1] or null; first, c0, c1: slots[threadIdx.x]
// and cu[threadIdx.x], cu[threadIdx.x + 1], read ahead by the caller so that the readings travel together.
// Holds __syncthreads: called by all threads.
struct Gate {
  int quit, bad, back;
};
__device__ __forceinline__ bool pass(const int32_t* slots, int n, int first, const KvDims& d,
                                     uint32_t* seen, Gate* g, int32_t* err, const int32_t* cu = nullptr,
                                     int c0 = 0, int c1 = 0) {
  if (threadIdx.x == 0) {
    g->quit = device_error_set(err) ? 1 : 0;
    g->bad = g->back = 0;
  }
  for (int i = threadIdx.x; i < (d.slots + 31) / 32; i += blockDim.x) seen[i] = 0u;
  __syncthreads();
  if (g->quit) return false;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int s = i == static_cast<int>(threadIdx.x) ? first : slots[i];
    if (s < 0 || s >= d.slots || ((atomicOr(&seen[s >> 5], 1u << (s & 31)) >> (s & 31)) & 1u)) g->bad = 1;
    if (cu && (i == static_cast<int>(threadIdx.x) ? c1 < c0 : cu[i + 1] < cu[i])) g->back = 1;
  }
  __syncthreads();
  if ((g->bad || g->back) && threadIdx.x == 0) set_device_error(err, g->bad ? RPP_DERR_SLOT : RPP_DERR_LENGTH);
  return !g->bad && !g->back;
}

// One reading of the error word for the whole CTA.
__device__ __forceinline__ bool quit(const int32_t* err, int* s_flag) {
  if (threadIdx.x == 0) *s_flag = device_error_set(err) ? 1 : 0;
  __syncthreads();
  return *s_flag != 0;
}

inline int blocks_for(long long work, int most) {
  if (work < 1) work = 1;
  return static_cast<int>(work < most ? work : most);
}

}  // namespace

}  // namespace rpp
