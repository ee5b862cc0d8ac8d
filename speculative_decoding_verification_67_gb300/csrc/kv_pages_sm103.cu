// Pages of the key-value cache: release, fork, reserve (copy on write) and
// compaction.  Declared in include/spec_kv_pages.h.
//
// The state is the block table and a count per page; a page is free iff its
// count is 0 and allocation takes the lowest free ids, so no free list has to
// be kept in order.
//
//  * release and fork touch rows of the table only: one warp per sequence,
//    one CTA per pair, each checking its row before it changes anything.
//  * reserve plans in one CTA (what each sequence needs, an exclusive scan,
//    the lowest free pages by ballots over the counts, the new entries) and
//    copies the shared partial pages with a dependent grid, one warp per 4 KB
//    piece of (sequence, layer).  A thread walks the columns of a sequence's
//    range, which suits a round's few positions: room for one prompt of 12301
//    tokens takes 242 us on pages of 16 and 3.8 ms on pages of one.
//  * compact plans in one CTA (live count, ordered lists of holes and of
//    pages to move) and moves pages and entries with a dependent grid.
//
// The plans are bound by latency: a handful of dependent passes over L2 by
// one CTA (reserve: for each column of the longest range).  The copies are
// bound by HBM: every moved byte is read once and written once.
#include <cstdint>

#include "internal.h"
#include "kv_copy.cuh"
#include "sm103_ptx.cuh"
#include "spec_kv_pages.h"

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kCopyWarps = kCopyThreads / 32;
constexpr int kCopyCtasPerSm = 8;
constexpr int kPieceVecs = 256;          // 16-byte vectors of one copy piece (4 KB)
constexpr int kScanWords = 16;           // words of 32 pages a warp looks at in one scan step
constexpr int kScanPages = kPlanWarps * kScanWords * 32;

struct PagesArgs {
  int32_t* seq_len;
  int32_t* bt;
  int32_t* ref;
  int B, max_pages, num_pages, page_size;
  int* ctrl;
  // plan arrays of the workspace
  int* off;      // [B] rank of the first page a sequence is given; -1 where it is not served
  int4* jobs;    // [B] (old page, new page, slots to copy, -)
  int* cnt;      // [num_pages] entries of the call's write ranges that name a page
  long long* last;  // [num_pages] the last of them, sequence (upper half) and column
  int* list;     // [num_pages] pages handed out / holes
  int* olds;     // [num_pages] page replaced by the k-th one handed out, or -1 / pages that move
  // copies
  uint4* pool;
  int layers;
  long long page_vecs, entry_vecs;
};

__device__ __forceinline__ int* row_of(const PagesArgs& a, int b) {
  return a.bt + static_cast<long long>(b) * a.max_pages;
}

// ------------------------------------------------------------------ release
__global__ void __launch_bounds__(kRowThreads) kv_release_kernel(const PagesArgs a, const int32_t* new_len) {
  const int lane = threadIdx.x & 31;
  int bits = 0;
  for (int b = blockIdx.x * kRowWarps + (threadIdx.x >> 5); b < a.B; b += gridDim.x * kRowWarps) {
    const int L = a.seq_len[b];
    const int to = new_len ? new_len[b] : L;
    if (to < 0 && new_len) continue;
    if (L < 0 || to > L) {
      bits |= SPEC_KV_DEVERR_LENGTH;
      continue;
    }
    int* row = row_of(a, b);
    const int c0 = to / a.page_size + (to % a.page_size != 0);
    int bad = 0;
    for (long long c = c0 + lane; c < a.max_pages; c += 32) {
      const int p = row[c];
      if (p >= a.num_pages) bad |= SPEC_KV_DEVERR_PAGE;
      else if (p >= 0 && a.ref[p] < 1) bad |= SPEC_KV_DEVERR_REF;
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (bad) {
      bits |= bad;
      continue;
    }
    for (long long c = c0 + lane; c < a.max_pages; c += 32) {
      const int p = row[c];
      if (p < 0) continue;
      if (atomicSub(a.ref + p, 1) < 1) {  // more holders than the count says: put it back
        atomicAdd(a.ref + p, 1);
        bits |= SPEC_KV_DEVERR_REF;
      }
      row[c] = -1;
    }
    __syncwarp();
    if (lane == 0) a.seq_len[b] = to;
  }
  if (bits) atomicOr(a.ctrl + sv::kKvCollect, bits);
  __syncthreads();
  if (threadIdx.x == 0 && sv::kv_last_cta(a.ctrl)) sv::kv_publish(a.ctrl);
}

// --------------------------------------------------------------------- fork
__global__ void __launch_bounds__(kRowThreads)
    kv_fork_kernel(const PagesArgs a, const int32_t* src, const int32_t* dst, int n) {
  const int i = blockIdx.x;
  const int s = src[i], d = dst[i];
  int bad = 0;
  if (s < 0 || s >= a.B || d < 0 || d >= a.B || s == d) bad = SPEC_KV_DEVERR_PAIR;
  // an earlier pair with this destination, or any pair whose destination is this source
  for (int k = threadIdx.x; k < n; k += kRowThreads) {
    const int dk = dst[k];
    if (dk == s || (dk == d && k < i)) bad = SPEC_KV_DEVERR_PAIR;
  }
  if (__syncthreads_or(bad)) bad = SPEC_KV_DEVERR_PAIR;
  int L = 0, used = 0;
  if (!bad) {
    L = a.seq_len[s];
    if (L < 0) bad = SPEC_KV_DEVERR_LENGTH;
    else if ((used = L / a.page_size + (L % a.page_size != 0)) > a.max_pages) bad = SPEC_KV_DEVERR_CAPACITY;
  }
  if (!bad) {
    const int* from = row_of(a, s);
    const int* to = row_of(a, d);
    for (long long c = threadIdx.x; c < a.max_pages; c += kRowThreads) {
      if (to[c] >= 0) bad |= SPEC_KV_DEVERR_BUSY;
      if (c >= used) continue;
      const int p = from[c];
      if (p < 0 || p >= a.num_pages) bad |= SPEC_KV_DEVERR_PAGE;
      else if (a.ref[p] < 1) bad |= SPEC_KV_DEVERR_REF;
    }
  }
  // every thread's bits: the sequence is copied only when none is set
  __shared__ int s_bad;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  if (bad) atomicOr(&s_bad, bad);
  __syncthreads();
  if (s_bad == 0) {
    const int* from = row_of(a, s);
    int* to = row_of(a, d);
    for (long long c = threadIdx.x; c < a.max_pages; c += kRowThreads) {
      int p = -1;
      if (c < used) {
        p = from[c];
        atomicAdd(a.ref + p, 1);
      }
      to[c] = p;
    }
    if (threadIdx.x == 0) a.seq_len[d] = L;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    if (s_bad) atomicOr(a.ctrl + sv::kKvCollect, s_bad);
    if (sv::kv_last_cta(a.ctrl)) sv::kv_publish(a.ctrl);
  }
}

// ------------------------------------------------------------ block-wide scan
// Exclusive scan of one value per thread over the CTA; `total` is the sum.
template <typename T>
__device__ T block_scan(T v, T* warp_sum, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T t = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    warp_sum[lane] = t;
  }
  __syncthreads();
  total = warp_sum[kPlanWarps - 1];
  const T before = warp == 0 ? T(0) : warp_sum[warp - 1];
  __syncthreads();
  return before + x - v;
}

// Appends the pages of [first, end) whose count is (or is not) positive to
// `list` in ascending order, stopping after `want` of them; returns how many
// were found (at most `want` are written).  All threads of the plan CTA.
__device__ int collect_pages(const int* ref, int first, int end, bool live, int want, int* list, long long* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int have = 0;
  for (long long p0 = first; p0 < end && have < want; p0 += kScanPages) {
    unsigned word[kScanWords];
    int mine = 0;
#pragma unroll
    for (int w = 0; w < kScanWords; ++w) {
      const long long p = p0 + (warp * kScanWords + w) * 32 + lane;
      word[w] = __ballot_sync(0xffffffffu, p < end && (ref[p] > 0) == live);
      mine += __popc(word[w]);
    }
    long long total;
    int at = have + static_cast<int>(block_scan(lane == 0 ? static_cast<long long>(mine) : 0ll, warp_sum, total));
    at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
    for (int w = 0; w < kScanWords; ++w) {
      if (word[w] >> lane & 1u) {
        const int k = at + __popc(word[w] & ((1u << lane) - 1u));
        if (k < want) list[k] = static_cast<int>(p0 + (warp * kScanWords + w) * 32 + lane);
      }
      at += __popc(word[w]);
    }
    have += static_cast<int>(total);
  }
  __syncthreads();  // the list is visible to the CTA
  return have < want ? have : want;
}

// ------------------------------------------------------------------ reserve
__device__ __forceinline__ long long entry_key(int b, int c) { return static_cast<long long>(b) << 32 | c; }

// Whether entry p in column c of the sequence's write range is replaced by a new page.
__device__ __forceinline__ bool replaced(const PagesArgs& a, int p, int b, int c) {
  if (p < 0) return true;
  const int r = a.ref[p];
  return r > 1 && !(a.cnt[p] >= r && a.last[p] == entry_key(b, c));
}

__global__ void __launch_bounds__(kPlanThreads) kv_reserve_kernel(const PagesArgs a, const int32_t* num_new) {
  __shared__ long long warp_sum[kPlanWarps];
  __shared__ int s_err;
  sv::griddep_launch_dependents();  // the copies may launch; they wait for this grid to finish
  if (threadIdx.x == 0) s_err = 0;
  __syncthreads();
  // what each sequence asks for, checked; the pages it writes start at no writer
  for (int b = threadIdx.x; b < a.B; b += kPlanThreads) {
    const int n = num_new[b], L = a.seq_len[b];
    int bad = 0, ok = 0;
    if (n < 0 || (n > 0 && L < 0)) bad = SPEC_KV_DEVERR_LENGTH;
    else if (n > 0) {
      const int c0 = L / a.page_size;
      const long long c1 = (static_cast<long long>(L) + n - 1) / a.page_size;
      if (c1 >= a.max_pages) bad = SPEC_KV_DEVERR_CAPACITY;
      else {
        const int* row = row_of(a, b);
        for (int c = c0; c <= c1; ++c) {
          const int p = row[c];
          if (p >= a.num_pages || (p < 0 && c == c0 && L % a.page_size)) bad |= SPEC_KV_DEVERR_PAGE;
          else if (p >= 0 && a.ref[p] < 1) bad |= SPEC_KV_DEVERR_REF;
        }
        if (!bad) {
          ok = 1;
          for (int c = c0; c <= c1; ++c) {
            const int p = row[c];
            if (p >= 0) {
              a.cnt[p] = 0;
              a.last[p] = -1;
            }
          }
        }
      }
    }
    if (bad) atomicOr(&s_err, bad);
    a.off[b] = ok ? 0 : -1;
    a.jobs[b] = make_int4(-1, -1, 0, 0);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < a.B; b += kPlanThreads) {
    if (a.off[b] < 0) continue;
    const int L = a.seq_len[b], c1 = (L + num_new[b] - 1) / a.page_size;
    const int* row = row_of(a, b);
    for (int c = L / a.page_size; c <= c1; ++c) {
      const int p = row[c];
      if (p >= 0) {
        atomicAdd(a.cnt + p, 1);
        atomicMax(a.last + p, entry_key(b, c));
      }
    }
  }
  __syncthreads();
  // pages needed, by ascending sequence (64 bits: a corrupt request may ask for more than 2^31)
  long long want = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    long long need = 0, total;
    const bool ok = b < a.B && a.off[b] >= 0;
    if (ok) {
      const int L = a.seq_len[b], c1 = (L + num_new[b] - 1) / a.page_size;
      const int* row = row_of(a, b);
      for (int c = L / a.page_size; c <= c1; ++c) need += replaced(a, row[c], b, c);
    }
    const long long at = want + block_scan(need, warp_sum, total);
    if (ok) a.off[b] = static_cast<int>(at < a.num_pages ? at : a.num_pages);  // beyond the pool: refused below
    want += total;
  }
  int found = 0;
  if (want <= a.num_pages) found = collect_pages(a.ref, 0, a.num_pages, false, static_cast<int>(want), a.list, warp_sum);
  if (found < want) {  // (uniform) nothing changes
    if (threadIdx.x == 0) {
      a.ctrl[sv::kKvErr] = s_err | SPEC_KV_DEVERR_POOL;
      a.ctrl[sv::kKvCount] = 0;
    }
    return;
  }
  for (int b = threadIdx.x; b < a.B; b += kPlanThreads) {
    int k = a.off[b];
    if (k < 0) continue;
    const int L = a.seq_len[b], c0 = L / a.page_size, c1 = (L + num_new[b] - 1) / a.page_size;
    int* row = row_of(a, b);
    for (int c = c0; c <= c1; ++c) {
      const int p = row[c];
      if (!replaced(a, p, b, c)) continue;  // counts of held pages change only after this loop
      const int q = a.list[k];
      a.olds[k++] = p;
      row[c] = q;
      if (p >= 0 && c == c0 && L % a.page_size) a.jobs[b] = make_int4(p, q, L % a.page_size, 0);
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < found; k += kPlanThreads) {
    a.ref[a.list[k]] = 1;
    if (a.olds[k] >= 0) atomicSub(a.ref + a.olds[k], 1);
  }
  if (threadIdx.x == 0) {
    a.ctrl[sv::kKvErr] = s_err;
    a.ctrl[sv::kKvCount] = 1;
  }
}

__global__ void __launch_bounds__(kCopyThreads) kv_reserve_copy_kernel(const PagesArgs a) {
  sv::griddep_wait();
  if (a.ctrl[sv::kKvCount] == 0) return;
  const int lane = threadIdx.x & 31;
  const long long pieces = (a.page_vecs + kPieceVecs - 1) / kPieceVecs;
  const long long units = static_cast<long long>(a.B) * a.layers * pieces;
  const long long plane = static_cast<long long>(a.num_pages) * a.page_vecs;
  for (long long u = static_cast<long long>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<long long>(gridDim.x) * kCopyWarps) {
    const int b = static_cast<int>(u / (pieces * a.layers));
    const int4 job = a.jobs[b];
    const long long v0 = (u % pieces) * kPieceVecs;
    long long n = job.z * a.entry_vecs - v0;
    if (n <= 0) continue;
    if (n > kPieceVecs) n = kPieceVecs;
    const long long layer = u / pieces % a.layers;
    sv::warp_copy(a.pool + layer * plane + job.x * a.page_vecs + v0, a.pool + layer * plane + job.y * a.page_vecs + v0, n,
                  lane);
  }
}

// ------------------------------------------------------------------ compact
__global__ void __launch_bounds__(kPlanThreads) kv_compact_kernel(const PagesArgs a, int32_t* out_num_live) {
  __shared__ long long warp_sum[kPlanWarps];
  __shared__ int s_err;
  sv::griddep_launch_dependents();
  if (threadIdx.x == 0) s_err = 0;
  __syncthreads();
  // where each page's entries go (cnt serves as the map): to the page itself, or -1 for a free one
  long long mine = 0, sum;
  for (long long p = threadIdx.x; p < a.num_pages; p += kPlanThreads) {
    const int r = a.ref[p];
    mine += r > 0;
    a.cnt[p] = r > 0 ? static_cast<int>(p) : -1;
    if (r < 0) atomicOr(&s_err, SPEC_KV_DEVERR_REF);
  }
  block_scan(mine, warp_sum, sum);
  const int live = static_cast<int>(sum);
  const int holes = collect_pages(a.ref, 0, live, false, live, a.list, warp_sum);
  collect_pages(a.ref, live, a.num_pages, true, holes, a.olds, warp_sum);
  for (int k = threadIdx.x; k < holes; k += kPlanThreads) {
    const int to = a.list[k], from = a.olds[k];  // (a hole's own place in the map stays -1)
    a.cnt[from] = to;
    a.ref[to] = a.ref[from];
    a.ref[from] = 0;
  }
  if (threadIdx.x == 0) {
    a.ctrl[sv::kKvErr] = s_err;
    a.ctrl[sv::kKvCount] = holes;
    if (out_num_live) *out_num_live = live;
  }
}

__global__ void __launch_bounds__(kCopyThreads) kv_compact_copy_kernel(const PagesArgs a) {
  sv::griddep_wait();
  const int moves = a.ctrl[sv::kKvCount];
  // block-table entries
  const long long cells = static_cast<long long>(a.B) * a.max_pages;
  int bits = 0;
  for (long long c = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; c < cells;
       c += static_cast<long long>(gridDim.x) * kCopyThreads) {
    const int p = a.bt[c];
    if (p < 0) continue;
    const int to = p < a.num_pages ? a.cnt[p] : -1;
    if (to < 0) bits |= SPEC_KV_DEVERR_PAGE;
    else if (to != p) a.bt[c] = to;
  }
  if (bits) atomicOr(a.ctrl + sv::kKvErr, bits);
  // contents
  const int lane = threadIdx.x & 31;
  const long long pieces = (a.page_vecs + kPieceVecs - 1) / kPieceVecs;
  const long long units = static_cast<long long>(moves) * a.layers * pieces;
  const long long plane = static_cast<long long>(a.num_pages) * a.page_vecs;
  for (long long u = static_cast<long long>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<long long>(gridDim.x) * kCopyWarps) {
    const long long v0 = (u % pieces) * kPieceVecs;
    const long long n = a.page_vecs - v0 < kPieceVecs ? a.page_vecs - v0 : kPieceVecs;
    const long long k = u / pieces % moves, layer = u / (pieces * moves);
    sv::warp_copy(a.pool + layer * plane + a.olds[k] * a.page_vecs + v0,
                  a.pool + layer * plane + a.list[k] * a.page_vecs + v0, n, lane);
  }
}

// --------------------------------------------------------------------- host
bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

bool dims_ok(const spec_kv_pages_dims& d) {
  return d.B >= 1 && d.B <= 65535 && d.max_pages >= 1 && d.num_pages >= 1 && d.page_size >= 1 &&
         static_cast<long long>(d.max_pages) * d.page_size < (1ll << 31) &&
         static_cast<long long>(d.num_pages) * d.page_size < (1ll << 31);
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

size_t workspace_size(const spec_kv_pages_dims& d) {
  return sv::kKvCtrlBytes + up(4 * static_cast<size_t>(d.B)) + up(16 * static_cast<size_t>(d.B)) +
         3 * up(4 * static_cast<size_t>(d.num_pages)) + up(8 * static_cast<size_t>(d.num_pages));
}

spec_status make_args(PagesArgs& a, int32_t* seq_len, int32_t* bt, int32_t* ref, const spec_kv_pages_dims& d, void* ws,
                      size_t bytes) {
  if (!bt || !ref || !ws) return SPEC_ERR_ARG;
  if (!dims_ok(d)) return SPEC_ERR_DIMS;
  if (misaligned(ws, 16) || misaligned(seq_len, 4) || misaligned(bt, 4) || misaligned(ref, 4)) return SPEC_ERR_ALIGN;
  if (bytes < workspace_size(d)) return SPEC_ERR_WORKSPACE;
  a = PagesArgs{};
  a.seq_len = seq_len;
  a.bt = bt;
  a.ref = ref;
  a.B = d.B;
  a.max_pages = d.max_pages;
  a.num_pages = d.num_pages;
  a.page_size = d.page_size;
  a.ctrl = static_cast<int*>(ws);
  char* p = static_cast<char*>(ws) + sv::kKvCtrlBytes;
  a.off = reinterpret_cast<int*>(p);
  p += up(4 * static_cast<size_t>(d.B));
  a.jobs = reinterpret_cast<int4*>(p);
  p += up(16 * static_cast<size_t>(d.B));
  a.last = reinterpret_cast<long long*>(p);
  p += up(8 * static_cast<size_t>(d.num_pages));
  for (int** q : {&a.cnt, &a.list, &a.olds}) {
    *q = reinterpret_cast<int*>(p);
    p += up(4 * static_cast<size_t>(d.num_pages));
  }
  return SPEC_OK;
}

spec_status pool_args(PagesArgs& a, void* pool, int32_t layers, int64_t entry_bytes) {
  if (layers < 1 || layers > 65535 || entry_bytes < 16 || entry_bytes % 16 != 0) return SPEC_ERR_DIMS;
  if (static_cast<double>(layers) * a.num_pages * a.page_size * static_cast<double>(entry_bytes) > 9.0e18)
    return SPEC_ERR_DIMS;
  if (misaligned(pool, 16)) return SPEC_ERR_ALIGN;
  a.pool = static_cast<uint4*>(pool);
  a.layers = layers;
  a.entry_vecs = entry_bytes / 16;
  a.page_vecs = a.entry_vecs * a.page_size;
  return SPEC_OK;
}

unsigned copy_grid(const PagesArgs& a, long long jobs, const sv::DeviceInfo& dev) {
  const double pieces = static_cast<double>((a.page_vecs + kPieceVecs - 1) / kPieceVecs);
  const double want = static_cast<double>(jobs) * a.layers * pieces / kCopyWarps + 1;
  const double cap = static_cast<double>(dev.sm_count) * kCopyCtasPerSm;
  return static_cast<unsigned>(want < cap ? want : cap);
}

spec_status launched() { return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

}  // namespace

extern "C" {

size_t spec_kv_pages_workspace_bytes(spec_kv_pages_dims dims) { return dims_ok(dims) ? workspace_size(dims) : 0; }

spec_status spec_kv_release(const int32_t* new_len, int32_t* seq_len, int32_t* block_table, int32_t* ref_count,
                            spec_kv_pages_dims dims, void* workspace, size_t workspace_bytes, spec_stream_t stream) {
  if (!seq_len) return SPEC_ERR_ARG;
  PagesArgs a;
  spec_status st = make_args(a, seq_len, block_table, ref_count, dims, workspace, workspace_bytes);
  if (st != SPEC_OK) return st;
  if (misaligned(new_len, 4)) return SPEC_ERR_ALIGN;
  sv::DeviceInfo dev;
  if ((st = static_cast<spec_status>(sv::current_device(dev))) != SPEC_OK) return st;
  const int want = (dims.B + kRowWarps - 1) / kRowWarps, cap = dev.sm_count * 8;
  kv_release_kernel<<<want < cap ? want : cap, kRowThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a, new_len);
  return launched();
}

spec_status spec_kv_fork(const int32_t* src, const int32_t* dst, int32_t n, int32_t* seq_len, int32_t* block_table,
                         int32_t* ref_count, spec_kv_pages_dims dims, void* workspace, size_t workspace_bytes,
                         spec_stream_t stream) {
  if (!seq_len || !src || !dst) return SPEC_ERR_ARG;
  PagesArgs a;
  spec_status st = make_args(a, seq_len, block_table, ref_count, dims, workspace, workspace_bytes);
  if (st != SPEC_OK) return st;
  if (n < 1 || n > 65535) return SPEC_ERR_DIMS;
  if (misaligned(src, 4) || misaligned(dst, 4)) return SPEC_ERR_ALIGN;
  sv::DeviceInfo dev;
  if ((st = static_cast<spec_status>(sv::current_device(dev))) != SPEC_OK) return st;
  kv_fork_kernel<<<n, kRowThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a, src, dst, n);
  return launched();
}

spec_status spec_kv_reserve(const int32_t* num_new, const int32_t* seq_len, int32_t* block_table, int32_t* ref_count,
                            void* pool, int32_t layers, int64_t entry_bytes, spec_kv_pages_dims dims, void* workspace,
                            size_t workspace_bytes, spec_stream_t stream) {
  if (!num_new || !seq_len || !pool) return SPEC_ERR_ARG;
  PagesArgs a;
  spec_status st =
      make_args(a, const_cast<int32_t*>(seq_len), block_table, ref_count, dims, workspace, workspace_bytes);
  if (st != SPEC_OK) return st;
  if ((st = pool_args(a, pool, layers, entry_bytes)) != SPEC_OK) return st;
  if (misaligned(num_new, 4)) return SPEC_ERR_ALIGN;
  sv::DeviceInfo dev;
  if ((st = static_cast<spec_status>(sv::current_device(dev))) != SPEC_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  kv_reserve_kernel<<<1, kPlanThreads, 0, s>>>(a, num_new);
  if ((st = launched()) != SPEC_OK) return st;
  if (sv::launch_dependent(kv_reserve_copy_kernel, dim3(copy_grid(a, dims.B, dev)), dim3(kCopyThreads), s, a) !=
      cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

spec_status spec_kv_compact(int32_t* block_table, int32_t* ref_count, void* pool, int32_t layers, int64_t entry_bytes,
                            int32_t* out_num_live, spec_kv_pages_dims dims, void* workspace, size_t workspace_bytes,
                            spec_stream_t stream) {
  if (!pool) return SPEC_ERR_ARG;
  PagesArgs a;
  spec_status st = make_args(a, nullptr, block_table, ref_count, dims, workspace, workspace_bytes);
  if (st != SPEC_OK) return st;
  if ((st = pool_args(a, pool, layers, entry_bytes)) != SPEC_OK) return st;
  if (misaligned(out_num_live, 4)) return SPEC_ERR_ALIGN;
  sv::DeviceInfo dev;
  if ((st = static_cast<spec_status>(sv::current_device(dev))) != SPEC_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  kv_compact_kernel<<<1, kPlanThreads, 0, s>>>(a, out_num_live);
  if ((st = launched()) != SPEC_OK) return st;
  const long long cells = static_cast<long long>(dims.B) * dims.max_pages;
  const unsigned by_pages = copy_grid(a, dims.num_pages / 2 + 1, dev);
  const long long by_cells = (cells + kCopyThreads - 1) / kCopyThreads;
  const long long cap = static_cast<long long>(dev.sm_count) * kCopyCtasPerSm;
  const long long grid = by_cells > by_pages ? (by_cells < cap ? by_cells : cap) : by_pages;
  if (sv::launch_dependent(kv_compact_copy_kernel, dim3(static_cast<unsigned>(grid)), dim3(kCopyThreads), s, a) !=
      cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

spec_status spec_kv_pages_read_error(void* workspace, int32_t* error_word, spec_stream_t stream) {
  if (!workspace || !error_word) return SPEC_ERR_ARG;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess ||
      cudaMemcpy(error_word, workspace, sizeof(int32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

}  // extern "C"
