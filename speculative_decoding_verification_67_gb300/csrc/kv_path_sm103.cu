// Commit of an accepted tree path into the paged cache.  Declared in
// include/spec_kv_pages.h.
//
// The kept entries (root, then the path) of one sequence are a list of
// (source row, destination row) pairs, the same in every layer.  A CTA takes
// one sequence and a share of the layers: it checks the path and looks its
// rows up once, into shared memory, and its warps then copy slices of 512
// bytes of one layer, all kept entries of a slice one after the other.
//
// In place, source and destination overlap.  The path ascends, so entry i
// moves down (L+i <= L+path[i-1]) and its destination is never the source of
// a later entry; one warp doing a slice's entries in ascending order, loads
// before stores, is therefore exact, and slices are independent.
//
// Bound by HBM (every kept byte read and written once) where the batch is
// large, by the dependent look-ups n -> path -> page -> entry (about 5 us in
// all) where it is small.
#include <cstdint>

#include "internal.h"
#include "kv_copy.cuh"
#include "spec_kv_pages.h"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxNodes = 256;
constexpr int kFlight = 4;

struct PathArgs {
  const int32_t* n;
  const int32_t* path;
  int32_t* seq_len;
  const int32_t* bt;
  const uint4* staged;  // null in place
  uint4* pool;
  int B, N, layers, page_size, num_pages, max_pages;
  long long entry_vecs;
  int* ctrl;
};

// The pool row of position pos of sequence b, or -1 with error bits set.
__device__ long long pool_row(const PathArgs& a, int b, long long pos, int& err) {
  const long long col = pos / a.page_size;
  if (col >= a.max_pages) {
    err |= SPEC_KV_DEVERR_CAPACITY;
    return -1;
  }
  const int page = a.bt[static_cast<long long>(b) * a.max_pages + col];
  if (page < 0 || page >= a.num_pages) {
    err |= SPEC_KV_DEVERR_PAGE;
    return -1;
  }
  return static_cast<long long>(page) * a.page_size + pos % a.page_size;
}

__global__ void __launch_bounds__(kThreads) kv_path_kernel(const PathArgs a) {
  __shared__ long long s_src[kMaxNodes], s_dst[kMaxNodes];
  __shared__ int s_err, s_last;
  const int b = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_err = 0;
  __syncthreads();
  const int n = a.n[b];
  const int L = a.seq_len[b];
  int keep = n < 0 ? 0 : n + 1;
  int err = 0;
  if (L < 0) err = SPEC_KV_DEVERR_LENGTH;
  else if (n >= a.N) err = SPEC_KV_DEVERR_PATH;
  else if (threadIdx.x < keep) {  // keep <= N <= 256 = kThreads
    const int i = threadIdx.x;
    const int32_t* path = a.path + static_cast<long long>(b) * a.N;
    const int node = i == 0 ? 0 : path[i - 1];
    const int before = i <= 1 ? 0 : path[i - 2];
    if (i > 0 && (node <= before || node >= a.N)) {
      err = SPEC_KV_DEVERR_PATH;
    } else {
      s_dst[i] = pool_row(a, b, static_cast<long long>(L) + i, err);
      s_src[i] = a.staged ? static_cast<long long>(b) * a.N + node
                          : pool_row(a, b, static_cast<long long>(L) + node, err);
    }
  }
  if (err) atomicOr(&s_err, err);
  __syncthreads();
  if (s_err) keep = 0;

  const long long slices = (a.entry_vecs + 31) / 32;
  const long long plane = static_cast<long long>(a.num_pages) * a.page_size * a.entry_vecs;
  const long long src_plane = a.staged ? static_cast<long long>(a.B) * a.N * a.entry_vecs : plane;
  const uint4* from = a.staged ? a.staged : a.pool;
  const int first = a.staged ? 0 : 1;  // in place the root is where it belongs
  if (keep > first) {
    // layers blockIdx.y, blockIdx.y + gridDim.y, ...
    const int mine = (a.layers - static_cast<int>(blockIdx.y) + static_cast<int>(gridDim.y) - 1) / gridDim.y;
    const long long units = slices * mine;
    for (long long u = warp; u < units; u += kWarps) {
      const long long layer = blockIdx.y + (u / slices) * static_cast<long long>(gridDim.y);
      const long long v = (u % slices) * 32 + lane;
      if (v >= a.entry_vecs) continue;  // (no warp-wide step below)
      const uint4* src = from + layer * src_plane + v;
      uint4* dst = a.pool + layer * plane + v;
      for (int i0 = first; i0 < keep; i0 += kFlight) {
        uint4 r[kFlight];
#pragma unroll
        for (int j = 0; j < kFlight; ++j)
          if (i0 + j < keep) r[j] = sv::ld_stream_16(src + s_src[i0 + j] * a.entry_vecs);
#pragma unroll
        for (int j = 0; j < kFlight; ++j)
          if (i0 + j < keep) dst[s_dst[i0 + j] * a.entry_vecs] = r[j];
      }
    }
  }

  // the last CTA advances the lengths (every CTA has read them); the CTAs of
  // blockIdx.y == 0 leave their sequence's count in the workspace for it
  if (threadIdx.x == 0 && blockIdx.y == 0) {
    reinterpret_cast<int*>(reinterpret_cast<char*>(a.ctrl) + sv::kKvCtrlBytes)[b] = keep;
    if (s_err) atomicOr(a.ctrl + sv::kKvCollect, s_err);
  }
  __syncthreads();
  if (threadIdx.x == 0) s_last = sv::kv_last_cta(a.ctrl);
  __syncthreads();
  if (!s_last) return;
  const volatile int* kept = reinterpret_cast<int*>(reinterpret_cast<char*>(a.ctrl) + sv::kKvCtrlBytes);
  for (int i = threadIdx.x; i < a.B; i += kThreads) a.seq_len[i] += kept[i];
  if (threadIdx.x == 0) sv::kv_publish(a.ctrl);
}

bool path_dims_ok(const spec_kv_dims& d) { return spec_kv_commit_workspace_bytes(d) != 0; }

size_t path_workspace(const spec_kv_dims& d) {
  return sv::kKvCtrlBytes + (sizeof(int) * static_cast<size_t>(d.B) + 255) / 256 * 256;
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

}  // namespace

extern "C" {

size_t spec_kv_path_workspace_bytes(spec_kv_dims dims) { return path_dims_ok(dims) ? path_workspace(dims) : 0; }

spec_status spec_kv_commit_path(const int32_t* num_accepted, const int32_t* path, int32_t* seq_len,
                                const int32_t* block_table, const void* staged, void* pool, spec_kv_dims dims,
                                void* workspace, size_t workspace_bytes, spec_stream_t stream) {
  if (!num_accepted || !path || !seq_len || !block_table || !pool || !workspace) return SPEC_ERR_ARG;
  if (!path_dims_ok(dims)) return SPEC_ERR_DIMS;
  if (misaligned(workspace, 16) || misaligned(pool, 16) || misaligned(staged, 16) || misaligned(num_accepted, 4) ||
      misaligned(path, 4) || misaligned(seq_len, 4) || misaligned(block_table, 4))
    return SPEC_ERR_ALIGN;
  if (workspace_bytes < path_workspace(dims)) return SPEC_ERR_WORKSPACE;
  sv::DeviceInfo dev;
  const int st = sv::current_device(dev);
  if (st != SPEC_OK) return static_cast<spec_status>(st);
  PathArgs a;
  a.n = num_accepted;
  a.path = path;
  a.seq_len = seq_len;
  a.bt = block_table;
  a.staged = static_cast<const uint4*>(staged);
  a.pool = static_cast<uint4*>(pool);
  a.B = dims.B;
  a.N = dims.S;
  a.layers = dims.layers;
  a.page_size = dims.page_size;
  a.num_pages = dims.num_pages;
  a.max_pages = dims.max_pages;
  a.entry_vecs = dims.entry_bytes / 16;
  a.ctrl = static_cast<int*>(workspace);
  // about eight CTAs per SM in all, at least one slice for every warp
  const long long slices = (a.entry_vecs + 31) / 32 * dims.layers;
  long long share = (static_cast<long long>(dev.sm_count) * 8 + dims.B - 1) / dims.B;
  if (share > (slices + kWarps - 1) / kWarps) share = (slices + kWarps - 1) / kWarps;
  if (share > dims.layers) share = dims.layers;
  if (share < 1) share = 1;
  kv_path_kernel<<<dim3(dims.B, static_cast<unsigned>(share)), kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      a);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
