// Pieces shared by the cache kernels that move whole entries: streaming
// 16-byte copies by one warp, and the ticket by which the last CTA of a grid
// publishes the call's error word.
#pragma once

#include <cstdint>

namespace sv {

// Control words at the start of a cache workspace (zeroed once by the
// caller): [0] error word of the latest call, [1] count, [2] ticket,
// [3] error bits collected by the running call.
enum { kKvErr = 0, kKvCount = 1, kKvTicket = 2, kKvCollect = 3 };
constexpr size_t kKvCtrlBytes = 256;

__device__ __forceinline__ uint4 ld_stream_16(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Copies vectors [0, n) with one warp, eight 512-byte loads in flight.
__device__ __forceinline__ void warp_copy(const uint4* src, uint4* dst, long long n, int lane) {
  constexpr int kFlight = 8;
  for (long long v0 = 0; v0 < n; v0 += 32 * kFlight) {
    uint4 r[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const long long v = v0 + lane + 32 * j;
      if (v < n) r[j] = ld_stream_16(src + v);
    }
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const long long v = v0 + lane + 32 * j;
      if (v < n) dst[v] = r[j];
    }
  }
}

// Called by one thread of every CTA after the CTA's error bits are in
// ctrl[kKvCollect] (atomicOr) and its other work is done: true in the last
// CTA, which has every other CTA's writes before it.
__device__ __forceinline__ bool kv_last_cta(int* ctrl) {
  __threadfence();
  const bool last = atomicAdd(reinterpret_cast<unsigned*>(ctrl + kKvTicket), 1u) == gridDim.x * gridDim.y - 1;
  if (last) __threadfence();
  return last;
}

// By one thread of the last CTA: the error word of this call; leaves the
// control words ready for the next.
__device__ __forceinline__ void kv_publish(int* ctrl) {
  ctrl[kKvErr] = atomicExch(ctrl + kKvCollect, 0);
  ctrl[kKvTicket] = 0;
}

}  // namespace sv
