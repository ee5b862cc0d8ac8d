// Attention over the paged cache and over packed prompts.  Declared in
// include/spec_attention.h.
//
// Simple form: one warp per (token, head).  Each lane holds head_dim / 32
// elements of the query and of the output; the warp walks the visible keys
// once with the running maximum and sum of the softmax, a dot product and its
// shuffle sum per key.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "internal.h"
#include "kv_copy.cuh"
#include "spec_attention.h"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTree = 256;

struct AttnArgs {
  const void* q;
  const void* k;          // pool, or packed keys
  const void* v;          // packed values
  const void* staged;
  const int32_t* bt;
  const int32_t* len;     // seq_len, or cu_q
  const int32_t* len_k;   // q_len (may be null), or cu_k
  const int32_t* parents;
  void* out;
  float* lse;
  float scale;
  int B, S, heads, kv_heads, page_size, num_pages, max_pages, total_q, total_k;
  long long q_stride, k_stride, v_stride;
  int* ctrl;
};

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(__half& y, float x) { y = __float2half_rn(x); }

// One sequence as the kernel sees it.
struct Seq {
  int Lq, Lk;           // queries, keys (new ones included)
  int q0;               // first row of q
  long long k0;         // first row of packed keys
  int err;
};

template <bool kPaged>
__device__ Seq sequence(const AttnArgs& a, int b, int lane) {
  Seq s;
  s.err = 0;
  if (kPaged) {
    const int L = a.len[b];
    const int n = a.len_k ? a.len_k[b] : a.S;
    s.Lq = n;
    s.q0 = b * a.S;
    s.k0 = 0;
    s.Lk = L + n;
    int err = 0;
    if (n < 0 || n > a.S) {
      err = SPEC_ATTN_DEVERR_LENGTH;
      s.Lq = a.S;
    } else if (L < 0) {
      err = SPEC_ATTN_DEVERR_LENGTH;
    } else if (n > 0) {
      const long long in_pool = static_cast<long long>(L) + (a.staged ? 0 : n);
      if (in_pool > static_cast<long long>(a.max_pages) * a.page_size) {
        err = SPEC_ATTN_DEVERR_CAPACITY;
      } else {
        for (long long c = lane; c * a.page_size < in_pool; c += 32) {
          const int p = a.bt[static_cast<long long>(b) * a.max_pages + c];
          if (p < 0 || p >= a.num_pages) err |= SPEC_ATTN_DEVERR_PAGE;
        }
        if (a.parents)
          for (int i = lane; i < n; i += 32) {
            const int p = a.parents[static_cast<long long>(b) * a.S + i];
            if (i == 0 ? p != -1 : (p < 0 || p >= i)) err |= SPEC_ATTN_DEVERR_TREE;
          }
      }
    }
    s.err = __reduce_or_sync(0xffffffffu, err);
  } else {
    const int a0 = a.len[b], a1 = a.len[b + 1], b0 = a.len_k[b], b1 = a.len_k[b + 1];
    s.Lq = a1 - a0;
    s.Lk = b1 - b0;
    s.q0 = a0;
    s.k0 = b0;
    if (a0 < 0 || a1 < a0 || a1 > a.total_q || b0 < 0 || b1 < b0 || b1 > a.total_k) {
      s.err = SPEC_ATTN_DEVERR_LENGTH;
      s.Lq = 0;
    }
  }
  return s;
}

template <typename T, int D, bool kPaged>
__global__ void __launch_bounds__(kThreads) attn_rows_kernel(const AttnArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y;
  const Seq s = sequence<kPaged>(a, b, lane);
  if (s.err && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.ctrl + sv::kKvCollect, s.err);
  const int G = a.heads / a.kv_heads;
  const long long entry = 2ll * a.kv_heads * D;
  for (long long r = static_cast<long long>(blockIdx.x) * kWarps + warp; r < static_cast<long long>(s.Lq) * a.heads;
       r += static_cast<long long>(gridDim.x) * kWarps) {
    const int i = static_cast<int>(r / a.heads), h = static_cast<int>(r % a.heads), g = h / G;
    const long long row = s.q0 + i;
    T* out = static_cast<T*>(a.out) + (row * a.heads + h) * D;
    float o[E], qf[E], m = -INFINITY, l = 0.f;
    const T* q = static_cast<const T*>(a.q) + row * a.q_stride + h * D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e] = 0.f;
      qf[e] = to_f(q[lane + 32 * e]);
    }
    if (!s.err) {
      const int L = s.Lk - s.Lq;       // keys before the first query (negative: fewer keys than queries)
      const int last = L + i;          // the last visible key of a chain
      // tree: the ancestors of i, as a bit per node (lane w: nodes 32w ..; at most 256 nodes)
      unsigned anc = 0;
      if (kPaged && a.parents)
        for (int p = i; p >= 0; p = a.parents[static_cast<long long>(b) * a.S + p])
          if (p / 32 == lane) anc |= 1u << (p % 32);
      for (int j = 0; j <= last; ++j) {
        const T *kp, *vp;
        if (kPaged) {
          if (j >= L && a.parents && !(__shfl_sync(0xffffffffu, anc, (j - L) / 32) >> ((j - L) % 32) & 1u)) continue;
          long long at;
          const T* base;
          if (a.staged && j >= L) {
            base = static_cast<const T*>(a.staged);
            at = static_cast<long long>(b) * a.S + (j - L);
          } else {
            base = static_cast<const T*>(a.k);
            at = static_cast<long long>(a.bt[static_cast<long long>(b) * a.max_pages + j / a.page_size]) * a.page_size +
                 j % a.page_size;
          }
          kp = base + at * entry + g * D;
          vp = kp + a.kv_heads * D;
        } else {
          kp = static_cast<const T*>(a.k) + (s.k0 + j) * a.k_stride + g * D;
          vp = static_cast<const T*>(a.v) + (s.k0 + j) * a.v_stride + g * D;
        }
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) dot += qf[e] * to_f(kp[lane + 32 * e]);
#pragma unroll
        for (int x = 16; x; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
        dot *= a.scale;
        const float top = fmaxf(m, dot);
        const float ref = top == -INFINITY ? 0.f : top;
        const float keep = expf(m - ref), w = expf(dot - ref);
        l = l * keep + w;
        m = top;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * to_f(vp[lane + 32 * e]);
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) from_f(out[lane + 32 * e], l == 0.f ? 0.f : o[e] * inv);
    if (a.lse && lane == 0) a.lse[row * a.heads + h] = l == 0.f ? -INFINITY : m + logf(l);
  }
  __syncthreads();
  if (threadIdx.x == 0 && sv::kv_last_cta(a.ctrl)) sv::kv_publish(a.ctrl);
}

// --------------------------------------------------------------------- host
bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

bool heads_ok(int heads, int kv_heads, int head_dim, int dtype) {
  return (head_dim == 64 || head_dim == 128) && kv_heads >= 1 && heads >= kv_heads && heads <= 1024 &&
         heads % kv_heads == 0 && heads / kv_heads <= 64 && (dtype == SPEC_ATTN_BF16 || dtype == SPEC_ATTN_FP16);
}

bool stride_ok(int64_t stride, int heads, int head_dim) {
  return stride % 8 == 0 && stride >= static_cast<int64_t>(heads) * head_dim && stride <= (1ll << 31);
}

constexpr int64_t kMaxTokens = 1 << 24;

bool kv_dims_ok(const spec_kv_attn_dims& d) {
  return heads_ok(d.heads, d.kv_heads, d.head_dim, d.dtype) && d.B >= 1 && d.B <= 65535 && d.S >= 1 &&
         d.S <= kMaxTree && static_cast<int64_t>(d.B) * d.S <= kMaxTokens && d.page_size >= 1 && d.num_pages >= 1 &&
         d.max_pages >= 1 && static_cast<int64_t>(d.max_pages) * d.page_size < (1ll << 31) &&
         static_cast<int64_t>(d.num_pages) * d.page_size < (1ll << 31) && stride_ok(d.q_stride, d.heads, d.head_dim);
}

bool prompt_dims_ok(const spec_prompt_dims& d) {
  return heads_ok(d.heads, d.kv_heads, d.head_dim, d.dtype) && d.B >= 1 && d.B <= 65535 && d.total_q >= 1 &&
         d.total_q <= kMaxTokens && d.total_k >= 1 && d.total_k <= kMaxTokens &&
         stride_ok(d.q_stride, d.heads, d.head_dim) && stride_ok(d.k_stride, d.kv_heads, d.head_dim) &&
         stride_ok(d.v_stride, d.kv_heads, d.head_dim);
}

size_t workspace_size() { return sv::kKvCtrlBytes; }

template <bool kPaged>
spec_status launch(const AttnArgs& a, int head_dim, int dtype, int rows, cudaStream_t s) {
  const long long warps = static_cast<long long>(rows) * a.heads;
  const long long want = (warps + kWarps - 1) / kWarps;
  const dim3 grid(static_cast<unsigned>(want < 4096 ? want : 4096), a.B);
  if (dtype == SPEC_ATTN_BF16) {
    if (head_dim == 64) attn_rows_kernel<__nv_bfloat16, 64, kPaged><<<grid, kThreads, 0, s>>>(a);
    else attn_rows_kernel<__nv_bfloat16, 128, kPaged><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (head_dim == 64) attn_rows_kernel<__half, 64, kPaged><<<grid, kThreads, 0, s>>>(a);
    else attn_rows_kernel<__half, 128, kPaged><<<grid, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t spec_kv_attention_workspace_bytes(spec_kv_attn_dims dims) { return kv_dims_ok(dims) ? workspace_size() : 0; }

size_t spec_prompt_attention_workspace_bytes(spec_prompt_dims dims) {
  return prompt_dims_ok(dims) ? workspace_size() : 0;
}

spec_status spec_kv_attention(const void* q, const void* pool, const int32_t* block_table, const int32_t* seq_len,
                              const void* staged, const int32_t* parents, const int32_t* q_len, float scale, void* out,
                              float* out_lse, spec_kv_attn_dims dims, void* workspace, size_t workspace_bytes,
                              spec_stream_t stream) {
  if (!q || !pool || !block_table || !seq_len || !out || !workspace) return SPEC_ERR_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SPEC_ERR_ARG;
  if (!kv_dims_ok(dims)) return SPEC_ERR_DIMS;
  if (misaligned(q, 16) || misaligned(pool, 16) || misaligned(staged, 16) || misaligned(out, 16) ||
      misaligned(workspace, 16) || misaligned(block_table, 4) || misaligned(seq_len, 4) || misaligned(parents, 4) ||
      misaligned(q_len, 4) || misaligned(out_lse, 4))
    return SPEC_ERR_ALIGN;
  if (workspace_bytes < workspace_size()) return SPEC_ERR_WORKSPACE;
  sv::DeviceInfo dev;
  const int st = sv::current_device(dev);
  if (st != SPEC_OK) return static_cast<spec_status>(st);
  AttnArgs a = {};
  a.q = q;
  a.k = pool;
  a.staged = staged;
  a.bt = block_table;
  a.len = seq_len;
  a.len_k = q_len;
  a.parents = parents;
  a.out = out;
  a.lse = out_lse;
  a.scale = scale;
  a.B = dims.B;
  a.S = dims.S;
  a.heads = dims.heads;
  a.kv_heads = dims.kv_heads;
  a.page_size = dims.page_size;
  a.num_pages = dims.num_pages;
  a.max_pages = dims.max_pages;
  a.q_stride = dims.q_stride;
  a.ctrl = static_cast<int*>(workspace);
  return launch<true>(a, dims.head_dim, dims.dtype, dims.S, reinterpret_cast<cudaStream_t>(stream));
}

spec_status spec_prompt_attention(const void* q, const void* k, const void* v, const int32_t* cu_q,
                                  const int32_t* cu_k, float scale, void* out, float* out_lse, spec_prompt_dims dims,
                                  void* workspace, size_t workspace_bytes, spec_stream_t stream) {
  if (!q || !k || !v || !cu_q || !out || !workspace) return SPEC_ERR_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SPEC_ERR_ARG;
  if (!prompt_dims_ok(dims)) return SPEC_ERR_DIMS;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(out, 16) || misaligned(workspace, 16) ||
      misaligned(cu_q, 4) || misaligned(cu_k, 4) || misaligned(out_lse, 4))
    return SPEC_ERR_ALIGN;
  if (workspace_bytes < workspace_size()) return SPEC_ERR_WORKSPACE;
  sv::DeviceInfo dev;
  const int st = sv::current_device(dev);
  if (st != SPEC_OK) return static_cast<spec_status>(st);
  AttnArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.len = cu_q;
  a.len_k = cu_k ? cu_k : cu_q;
  a.out = out;
  a.lse = out_lse;
  a.scale = scale;
  a.B = dims.B;
  a.heads = dims.heads;
  a.kv_heads = dims.kv_heads;
  a.total_q = dims.total_q;
  a.total_k = dims.total_k;
  a.q_stride = dims.q_stride;
  a.k_stride = dims.k_stride;
  a.v_stride = dims.v_stride;
  a.ctrl = static_cast<int*>(workspace);
  return launch<false>(a, dims.head_dim, dims.dtype, dims.total_q, reinterpret_cast<cudaStream_t>(stream));
}

spec_status spec_attention_read_error(void* workspace, int32_t* error_word, spec_stream_t stream) {
  if (!workspace || !error_word) return SPEC_ERR_ARG;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess ||
      cudaMemcpy(error_word, workspace, sizeof(int32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

}  // extern "C"
