// Draws from filtered distributions.  Declared in include/spec_sample.h.
//
// A cluster of CTAs serves a row; each keeps its slice of the logits in shared
// memory, so they are read from HBM once, whatever passes follow (what does not
// fit is read again, mostly from L2, through rings of asynchronous copies):
//   1. maximum and smallest finite value;
//   2. top-k: a histogram of counts over equal steps of z, the step in which the
//      k-th falls, and the order of the few tokens in it by comparison with one
//      another; top-p likewise, with weights beside the counts.  A step that
//      holds too many tokens (ties, outliers) is taken apart by the bits of z;
//   3. the kept weights' sums, warp by warp (a warp has consecutive ids), and the
//      draw: the CTA, the warp, and the token in which u S falls;
//   4. the filtered logits.
// What the cluster agrees on goes through distributed shared memory.
//
// Weights are integers: 2^(z c) with c = log2(e) / T as a float pair, its
// fraction split into 1/512ths (a table) and a remainder below 2^-10 (three
// terms of the series), gives 32 bits, shifted into 2^-46 of the largest.  Sums
// are exact, so masses found in any order agree, and a prefix is compared with
// top_p or u as a product of integers.  An f32 exponential would decide one
// draw in 10^4 of 10^5 tokens differently from 64-bit arithmetic.
//
// Bound by the instructions of the passes (a weight takes about 45) and the
// cluster's barriers, a dozen a row, not by HBM: 64 rows of 152064 without
// filters take 39 us (1.0 TB/s, issue slots 57 % busy), 256 rows of 128256
// with settings of their own 197, 40 filtered rows with their logits written
// 66, one row of 32000 18 (a call from Python).
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "kv_copy.cuh"
#include "sm103_ptx.cuh"
#include "spec_sample.h"

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512;        // two CTAs to an SM
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 512;           // tokens that are ordered by comparison
constexpr int kMaxCluster = 8;
constexpr int kFrame = 46;           // the largest weight is at most 2^kFrame
constexpr int kSharedBytes = 115712; // of a CTA, two to an SM (113 KB each)
constexpr int kStages = 4;           // 16-byte pieces that a thread has under way of what is read from memory again

struct Table {
  unsigned v[512];
};
// 2^(j/512) in units of 2^-31 (32 bits).
constexpr Table make_table() {
  Table t = {};
  for (int j = 0; j < 512; ++j) {
    const double x = j / 512.0 * 0.69314718055994530942;
    double term = 1.0, sum = 0.0;
    for (int i = 1; i < 26; ++i) {
      term *= x / i;
      sum += term;
    }
    t.v[j] = 2147483648u + static_cast<unsigned>(sum * 2147483648.0 + 0.5);
  }
  return t;
}
__device__ constexpr Table kTable = make_table();

struct SampleArgs {
  const float* z;
  const float* u;
  spec_sample_params par;
  int32_t* out_tokens;
  float* out_logits;
  int rows, V, cap;       // cap: floats of a slice held in shared memory
  int per;                // tokens of a CTA's slice (a multiple of 4)
  int seg;                // consecutive floats of the slice's place in shared memory to a warp (a multiple of 128)
  long long ld, out_ld;
  int* ctrl;
};

// What turns a logit into a weight.
struct Expo {
  float base, ch, cl;
  int k;
};

struct Shared {
  uint2 table[512];               // 2^(j/512) in units of 2^-31, as a whole number and in f32
  union {
    unsigned hist[2][kBins];      // of this CTA: counts, or sums of weights (low and high words)
    struct {                      // once they have been added up: the tokens to put in order
      uint4 list[kList];          // key, token, weight (low and high word)
    };
  };
  unsigned list_n;
  float warp_f[2][kWarps];
  unsigned warp_u[kWarps];
  u64 warp_m[kWarps];
  // [rank] what each CTA of the cluster says
  float all_max[kMaxCluster], all_min[kMaxCluster];
  unsigned all_bad[kMaxCluster], all_count[kMaxCluster];
  u64 all_mass[kMaxCluster];
  int pick_bin;
  u64 pick_before;                // count or mass of the bins before
  float cut_z;
  int cut_id;
  double log_min_p;
};

// ------------------------------------------------------- distributed memory
__device__ __forceinline__ void put_u32(uint32_t addr, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void put_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned get_u32(uint32_t addr) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ unsigned add_u32(uint32_t addr, unsigned x) {
  unsigned v;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(v) : "r"(addr), "r"(x) : "memory");
  return v;
}
__device__ __forceinline__ void add_u64(uint32_t addr, u64 x) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(addr), "l"(x) : "memory");
}
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int bytes) {
  if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t at(const void* p, int rank) { return sv::cluster_map(p, rank); }

// ------------------------------------------------------------------ weights
__device__ __forceinline__ u64 weight(float z, const Expo& c, const uint2* table) {
  const float x = z - c.base;
  float p = x * c.ch;
  const float e = fmaf(x, c.cl, fmaf(x, c.ch, -p));
  p = fmaxf(p, -8000.f);  // (far below what a weight can hold; also where z is -infinity)
  const float m = fmaf(p, 512.f, 12582912.f);  // 1.5 * 2^23: the nearest whole number of 1/512ths in the low bits
  const float r = fmaf(m - 12582912.f, -1.f / 512, p) + e;
  const float q = r * fmaf(r, fmaf(r, 0.0555041087f, 0.240226507f), 0.693147181f);  // 2^r - 1
  const int i = __float_as_int(m) - 0x4B400000;
  const uint2 t = table[i & 511];
  const unsigned w = t.x + (__float_as_int(fmaf(q, __uint_as_float(t.y), 12582912.f)) - 0x4B400000);  // (below 2^22)
  const int n = min(c.k - (i >> 9), 63);
  return ((static_cast<u64>(w) << (kFrame - 30)) >> n) + 1 >> 1;
}

// floor(x * whole / 2^24-ish) of a float x in [0, 1) and a whole number, and whether something is left.
__device__ __forceinline__ u64 share_of(float x, u64 whole, bool& rest) {
  const unsigned bits = __float_as_uint(x), ex = bits >> 23;
  const u64 man = ex ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int shift = 150 - static_cast<int>(ex ? ex : 1);  // x = man / 2^shift, shift >= 24
  const u64 lo = man * whole, hi = __umul64hi(man, whole);
  if (shift >= 128) {
    rest = (lo | hi) != 0;
    return 0;
  }
  if (shift >= 64) {
    const int s = shift - 64;
    rest = lo != 0 || (hi & ((1ull << s) - 1)) != 0;
    return hi >> s;
  }
  rest = (lo & ((1ull << shift) - 1)) != 0;
  return (hi << (64 - shift)) | (lo >> shift);
}

// Descending: the larger z, the smaller the key.
__device__ __forceinline__ unsigned key_of(float z) {
  const unsigned b = __float_as_uint(z + 0.f);  // (-0 as 0)
  return b & 0x80000000u ? b : ~(b | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned key) {
  return __uint_as_float(key & 0x80000000u ? key : ~key & 0x7fffffffu);
}
__device__ __forceinline__ bool kept_by(float z, int id, float cut_z, int cut_id) {
  return z > cut_z || (z == cut_z && id <= cut_id);
}

__device__ __forceinline__ u64 warp_sum(u64 x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ u64 warp_scan(u64 x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// The bins that a CTA of the cluster adds up (a pair at least: what follows them starts on 16 bytes).
__host__ __device__ constexpr int bins_of(int ranks) { return (kBins + 2 * ranks - 1) / (2 * ranks) * 2; }

struct Row {
  const SampleArgs& a;
  Shared& sh;
  float4* ring;            // shared, this thread's: [kStages] kThreads apart
  u64* sum;                // shared: the bins (of kBins / ranks) that this CTA adds up for the cluster (counts or masses)
  const float* slice;      // shared; the slice's first token lies `shift` floats in, as it lies in 16 bytes of memory
  const float* from;       // the slice in memory
  int begin, n;            // its first token, how many
  int shift;
  int rank, ranks;
  float zmax;
  Expo c;

  __device__ __forceinline__ float value(int i) const { return i + shift < a.cap ? slice[i + shift] : from[i]; }

  // f(i, z) for the slice's tokens, four at a time to a lane; a warp has consecutive ones.  All lanes call f (with z =
  // -infinity outside the slice).  What shared memory does not hold comes from memory (or L2) through a ring of the
  // thread's own.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    each4([&](int i, float4 v) {
      f(i, v.x);
      f(i + 1, v.y);
      f(i + 2, v.z);
      f(i + 3, v.w);
    });
  }
  template <typename F>
  __device__ __forceinline__ void each4(F f) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = warp * a.seg + 4 * lane, all = n + shift, end = min(all, (warp + 1) * a.seg);
    auto ask = [&](int b, int stage) {
      if (b + 4 > a.cap && b >= shift && b + 4 <= all && b < end)
        copy_async(sv::smem_u32(ring + stage * kThreads), from + (b - shift), 16);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (all > a.cap)
      for (int t = 0; t < kStages - 1; ++t) ask(first + 128 * t, t);
    int stage = 0;
#pragma unroll 1
    for (int b = first; b - 4 * lane < end; b += 128) {
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (all > a.cap) {
        ask(b + 128 * (kStages - 1), (stage + kStages - 1) % kStages);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      }
      if (b >= shift && b + 4 <= all) {
        v = *reinterpret_cast<const float4*>(b + 4 <= a.cap ? slice + b : reinterpret_cast<const float*>(ring + stage * kThreads));
      } else {  // the slice's ends
        if (b >= shift && b < all) v.x = value(b - shift);
        if (b + 1 >= shift && b + 1 < all) v.y = value(b + 1 - shift);
        if (b + 2 >= shift && b + 2 < all) v.z = value(b + 2 - shift);
        if (b + 3 >= shift && b + 3 < all) v.w = value(b + 3 - shift);
      }
      stage = (stage + 1) % kStages;
      f(b - shift, v);
    }
  }

  // The last kept token, in descending order, bounded by count (`k`) or by mass (`p`).  Tokens beyond (cut_z, cut_id),
  // from an earlier selection, do not take part.  Ends with sh.cut_z, sh.cut_id set in every CTA; false (in all of them)
  // where everything is kept.
  template <bool kMass>
  __device__ bool select(unsigned k, float p, float range, float cut_z, int cut_id) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float scale = fminf(kBins / (2.f * range), 1e30f) * 2.f;  // steps per unit of half of z
    const float top = 0.5f * zmax;
    auto step_of = [&](float z) {
      const float m = fmaf(top - 0.5f * z, scale, 12582912.f);
      return min(static_cast<unsigned>(__float_as_int(fminf(m, 12582912.f + kBins)) - 0x4B400000), kBins - 1u);
    };
    int level = 0;           // 0: steps of z; then 11, 11 and 10 bits of the key
    unsigned step = 0, prefix = 0;
    u64 before = 0, target = k;
    auto shift_of = [](int level) { return level == 1 ? 21 : level == 2 ? 10 : 0; };
    // whether a token is of the step and the digits found so far
    auto inside = [&](int id, float z) {
      if (!(z > -INFINITY) || !kept_by(z, id, cut_z, cut_id)) return false;
      if (level == 0) return true;
      return step_of(z) == step && (level == 1 || key_of(z) >> shift_of(level - 1) == prefix);
    };
    while (true) {
#pragma unroll 1
      for (int i = tid; i < kBins; i += kThreads) sh.hist[0][i] = sh.hist[1][i] = 0;
      __syncthreads();
      // four tokens at a time, so that their additions are under way together
      each4([&](int i, float4 v) {
        const float z[4] = {v.x, v.y, v.z, v.w};
        bool in[4];
        unsigned bin[4], lo[4], hi[4], old[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) in[e] = inside(begin + i + e, z[e]);
        if (!(in[0] || in[1] || in[2] || in[3])) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          bin[e] = level == 0 ? step_of(z[e]) : key_of(z[e]) >> shift_of(level) & (level == 3 ? 1023u : 2047u);
          const u64 w = kMass ? weight(z[e], c, sh.table) : 1;
          lo[e] = static_cast<unsigned>(w);
          hi[e] = static_cast<unsigned>(w >> 32);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) old[e] = in[e] ? atomicAdd(&sh.hist[0][bin[e]], lo[e]) : 0u;
        if (kMass) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const unsigned up = hi[e] + (old[e] + lo[e] < old[e] ? 1u : 0u);
            if (in[e] && up) atomicAdd(&sh.hist[1][bin[e]], up);
          }
        }
      });
      __syncthreads();
      // every CTA adds its bins to those of the CTA that has them
      const int per = bins_of(ranks);
#pragma unroll 1
      for (int i = tid; i < kBins; i += kThreads) {
        const u64 x = kMass ? sh.hist[0][i] + (static_cast<u64>(sh.hist[1][i]) << 32) : sh.hist[0][i];
        if (x) add_u64(at(&sum[i % per], i / per), x);
      }
      sv::cluster_sync();
      constexpr int kEach = (kBins + kThreads - 1) / kThreads;  // consecutive bins of a thread (one CTA: four)
      const int mine = (per + kThreads - 1) / kThreads;
      u64 x[kEach], total = 0;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int i = tid * mine + j;
        x[j] = j < mine && i < per ? sum[i] : 0;
        total += x[j];
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (j < mine && tid * mine + j < per) sum[tid * mine + j] = 0;  // (ready for the next level)
      const u64 scan = warp_scan(total, lane);
      if (lane == 31) sh.warp_m[warp] = scan;
      if (tid == 0) sh.list_n = 0;
      __syncthreads();
      u64 at_bin = scan - total, all = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at_bin += sh.warp_m[w];
        all += sh.warp_m[w];
      }
      if (tid < ranks) put_u64(at(&sh.all_mass[rank], tid), all);
      sv::cluster_sync();
      u64 everything = 0;
      for (int r = 0; r < ranks; ++r) {
        if (r < rank) at_bin += sh.all_mass[r];
        everything += sh.all_mass[r];
      }
      if (level == 0) {
        if (kMass) {
          bool rest = false;
          target = p > 0.f ? share_of(p, everything, rest) : 0;
          if (rest) ++target;  // a token is kept while the mass before it is below p S, so below ceil(p S)
          if (target == 0) target = 1;
        } else if (target >= everything) {
          sv::cluster_sync();  // (what has been read may be written again)
          return false;
        }
      }
      at_bin += before;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        if (x[j] != 0 && at_bin < target && target <= at_bin + x[j]) {
          for (int r = 0; r < ranks; ++r) {
            put_u32(at(&sh.pick_bin, r), rank * per + tid * mine + j);
            put_u64(at(&sh.pick_before, r), at_bin);
          }
        }
        at_bin += x[j];
      }
      sv::cluster_sync();
      const unsigned bin = sh.pick_bin;
      before = sh.pick_before;
      if (level == 0) step = bin;
      else prefix = level == 1 ? bin : prefix << (level == 3 ? 10 : 11) | bin;
      ++level;
      // ---- the bin's tokens, to the first CTA
      each([&](int i, float z) {
        if (!inside(begin + i, z)) return;
        u64 w = 0;
        if (kMass && (w = weight(z, c, sh.table)) == 0) return;
        const unsigned spot = add_u32(at(&sh.list_n, 0), 1u);
        if (spot >= kList) return;
        put_u64(at(&sh.list[spot].x, 0), static_cast<u64>(begin + i) << 32 | key_of(z));
        put_u64(at(&sh.list[spot].z, 0), kMass ? w : 1);
      });
      sv::cluster_sync();
      const unsigned many = get_u32(at(&sh.list_n, 0));
      if (many <= kList) {  // few enough to put in order by comparison
        if (rank == 0) {
          int share = 1;  // lanes to a token
          while (share < 32 && many * share * 2 <= kThreads) share *= 2;
          const int i = tid / share, sub = tid % share;
          const uint4 self = i < many ? sh.list[i] : make_uint4(0, 0, 0, 0);
          u64 ahead = 0;
          if (i < many) {
#pragma unroll 4
            for (unsigned j = sub; j < many; j += share) {
              const uint4 other = sh.list[j];
              if (other.x < self.x || (other.x == self.x && other.y < self.y))
                ahead += static_cast<u64>(other.w) << 32 | other.z;
            }
          }
          for (int o = share / 2; o; o >>= 1) ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
          ahead += before;
          // the last token that is kept
          if (i < many && sub == 0 && ahead < target && target <= ahead + (static_cast<u64>(self.w) << 32 | self.z)) {
            for (int r = 0; r < ranks; ++r) {
              put_u32(at(&sh.cut_z, r), __float_as_uint(value_of(self.x)));
              put_u32(at(&sh.cut_id, r), self.y);
            }
          }
        }
        sv::cluster_sync();
        return true;
      }
      sv::cluster_sync();  // (the count has been read everywhere)
      if (level == 4) {  // one value, too many equals
        resolve_ties<kMass>(target - before, prefix, cut_z, cut_id);
        return true;
      }
    }
  }

  // More equals than the list holds: the r-th of them by token id.
  template <bool kMass>
  __device__ void resolve_ties(u64 missing, unsigned key, float cut_z, int cut_id) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float z0 = value_of(key);
    const u64 w0 = kMass ? weight(z0, c, sh.table) : 1;
    const unsigned r = static_cast<unsigned>((missing + w0 - 1) / w0);
    unsigned mine = 0;
    each([&](int i, float z) { mine += z == z0 && kept_by(z, begin + i, cut_z, cut_id); });
#pragma unroll
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) sh.warp_u[warp] = mine;
    __syncthreads();
    unsigned before = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.warp_u[w];
      all += sh.warp_u[w];
    }
    if (tid < ranks) put_u32(at(&sh.all_count[rank], tid), all);
    sv::cluster_sync();
    for (int q = 0; q < rank; ++q) before += sh.all_count[q];
    if (before < r && r <= before + mine) {  // (one warp of one CTA)
      const int end = min(n + shift, (warp + 1) * a.seg);
      for (int b0 = warp * a.seg; b0 < end; b0 += 32) {
        const int b = b0 + lane, i = b - shift;
        const float z = b < end && i >= 0 ? value(i) : -INFINITY;
        const bool hit = z == z0 && kept_by(z, begin + i, cut_z, cut_id);
        const unsigned word = __ballot_sync(0xffffffffu, hit);
        if (hit && before + __popc(word & ((1u << lane) - 1u)) + 1 == r) {
          for (int q = 0; q < ranks; ++q) {
            put_u32(at(&sh.cut_z, q), __float_as_uint(z0));
            put_u32(at(&sh.cut_id, q), begin + i);
          }
        }
        before += __popc(word);
        if (before >= r) break;
      }
    }
    sv::cluster_sync();
  }
};

__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  float* slice = reinterpret_cast<float*>(raw + (sizeof(Shared) + 15) / 16 * 16);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned ranks;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int rank = sv::cluster_ctarank();
  const int row = blockIdx.x / ranks;
  u64* sum = reinterpret_cast<u64*>(slice + a.cap);
  Row w = {a, sh, reinterpret_cast<float4*>(sum + bins_of(ranks)) + tid, sum, slice, nullptr, rank * a.per, 0, 0, rank, static_cast<int>(ranks), 0.f, {}};
  w.n = max(0, min(a.per, a.V - w.begin));
  w.from = a.z + row * a.ld + w.begin;
  w.shift = static_cast<int>(reinterpret_cast<uintptr_t>(w.from) >> 2 & 3);

  // ---- the slice, all of it under way at once
  {
    const int end = min(w.n + w.shift, a.cap);
    for (int b = 4 * tid; b < end; b += 4 * kThreads) {
      if (b >= w.shift && b + 4 <= end) {
        copy_async(sv::smem_u32(slice + b), w.from + (b - w.shift), 16);
      } else {
        for (int e = max(b, w.shift); e < min(b + 4, end); ++e) copy_async(sv::smem_u32(slice + e), w.from + (e - w.shift), 4);
      }
    }
  }
  for (int i = tid; i < bins_of(ranks); i += kThreads) sum[i] = 0;
  static_assert(kThreads == 512, "a thread for each entry of the table");
  sh.table[tid] = make_uint2(kTable.v[tid], __float_as_uint(__uint2float_rn(kTable.v[tid])));
  const float min_p = a.par.min_ps ? a.par.min_ps[row] : a.par.min_p;
  if (tid == 0 && min_p > 0.f) sh.log_min_p = log(static_cast<double>(fminf(min_p, 1.f)));  // (one thread: 64-bit units are few)
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  // its extremes
  float most = -INFINITY, least = INFINITY;
  unsigned bad = 0;
  int first = 0x7fffffff;  // the lowest id of the thread's largest
  w.each([&](int i, float z) {
    bad |= !(z < INFINITY);  // NaN or +infinity
    if (z > most) first = w.begin + i;
    most = fmaxf(most, z);
    least = fminf(least, z > -INFINITY ? z : INFINITY);
  });
  const float own = most;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    sh.warp_f[0][warp] = most;
    sh.warp_f[1][warp] = least;
    sh.warp_u[warp] = bad;
  }
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) {
    most = fmaxf(most, sh.warp_f[0][i]);
    least = fminf(least, sh.warp_f[1][i]);
    bad |= sh.warp_u[i];
  }
  // (a CTA's shared memory is written by others only once all of the cluster run)
  sv::cluster_sync();
  if (tid < ranks) {
    put_u32(at(&sh.all_max[rank], tid), __float_as_uint(most));
    put_u32(at(&sh.all_min[rank], tid), __float_as_uint(least));
    put_u32(at(&sh.all_bad[rank], tid), bad);
  }
  sv::cluster_sync();
  for (int r = 0; r < w.ranks; ++r) {
    most = fmaxf(most, sh.all_max[r]);
    least = fminf(least, sh.all_min[r]);
    bad |= sh.all_bad[r];
  }
  w.zmax = most;
  float T = a.par.temperatures ? a.par.temperatures[row] : a.par.temperature;
  const int top_k = a.par.top_ks ? a.par.top_ks[row] : a.par.top_k;
  const float top_p = a.par.top_ps ? a.par.top_ps[row] : a.par.top_p;
  int err = bad || !(most > -INFINITY) ? SPEC_SAMPLE_DEVERR_NONFINITE : 0;
  if (!(T >= 0.f && T < INFINITY) || top_p != top_p || min_p != min_p) err |= SPEC_SAMPLE_DEVERR_PARAM;

  if (err) {
    if (rank == 0 && tid == 0 && a.out_tokens) a.out_tokens[row] = -1;
  } else {
    float cut_z = -INFINITY, floor_z = -INFINITY;  // kept: up to the cut, and at least floor_z
    int cut_id = 0x7fffffff;
    const bool greedy = T == 0.f;
    const float away = 512.f * (greedy ? 1.f : T);
    T = fminf(fmaxf(T, 7.8886091e-31f), 1.2676506e30f);
    if (greedy) {
      cut_z = most;
    } else {
      w.c.ch = 1.44269502f / T;  // log2(e) = 1.44269502 + 1.92596299e-8, divided to twice f32's precision
      w.c.cl = (fmaf(-w.c.ch, T, 1.44269502f) + 1.92596299e-8f) / T;
      // Large exponents: of differences to the maximum, exact for every logit whose weight is not 0.
      w.c.base = fabsf(most * w.c.ch) > 4096.f ? most : 0.f;
      w.c.k = static_cast<int>(ceilf((most - w.c.base) * w.c.ch)) + max(0, 32 - __clz(a.V - 1) - 17);
      if (min_p > 0.f)  // exp((z - most) / T) >= min_p
        floor_z = __double2float_ru(static_cast<double>(most) + sh.log_min_p * static_cast<double>(T));
      const float range = fmaxf(0.5f * most - 0.5f * least, 1e-37f);  // half of it
      if (top_k > 0 && w.select<false>(top_k, 0.f, range, -INFINITY, 0x7fffffff)) {
        cut_z = sh.cut_z;
        cut_id = sh.cut_id;
        sv::cluster_sync();  // (read before the next selection writes them)
      }
      if (top_p < 1.f) {
        // steps down to weights of 2^-47 only
        const float narrow = fminf(range, 0.5f * 48.f / w.c.ch);
        if (w.select<true>(0, top_p, narrow, cut_z, cut_id)) {
          cut_z = sh.cut_z;
          cut_id = sh.cut_id;
        }
      }
    }
    auto kept = [&](int i, float z) {
      return z > -INFINITY && z >= floor_z && kept_by(z, w.begin + i, cut_z, cut_id);
    };
    int token = -1;  // greedy: the lowest id, for the filtered logits
    if (greedy) {
      int id = __reduce_min_sync(0xffffffffu, own == most ? first : 0x7fffffff);
      if (lane == 0) sh.warp_u[warp] = id;
      __syncthreads();
      for (int i = 0; i < kWarps; ++i) id = min(id, static_cast<int>(sh.warp_u[i]));
      if (tid < ranks) put_u32(at(&sh.all_count[rank], tid), id);
      sv::cluster_sync();
      for (int r = 0; r < w.ranks; ++r) id = min(id, static_cast<int>(sh.all_count[r]));
      cut_id = token = id;
      if (rank == 0 && tid == 0 && a.out_tokens) a.out_tokens[row] = token;
    } else if (a.out_tokens) {
      // ---- the draw
      u64 sum = 0;
      if (cut_z == -INFINITY && floor_z == -INFINITY)
        w.each([&](int, float z) { sum += weight(z, w.c, sh.table); });  // (0 for -infinity)
      else
        w.each([&](int i, float z) {
          if (kept(i, z)) sum += weight(z, w.c, sh.table);
        });
      sum = warp_sum(sum);
      if (lane == 0) sh.warp_m[warp] = sum;
      __syncthreads();
      u64 all = 0;
      for (int i = 0; i < kWarps; ++i) all += sh.warp_m[i];
      if (tid < ranks) put_u64(at(&sh.all_mass[rank], tid), all);
      sv::cluster_sync();
      u64 total = 0, before = 0;
      for (int r = 0; r < w.ranks; ++r) {
        if (r < rank) before += sh.all_mass[r];
        total += sh.all_mass[r];
      }
      const float u = a.u[row];
      bool rest;
      u64 target = u >= 1.f ? total : (u > 0.f ? share_of(u, total, rest) : 0) + 1;  // the smallest C_v that will do
      if (target > total) target = total;
      if (before < target && target <= before + all) {  // (in one CTA)
        int s = 0;
        while (before + sh.warp_m[s] < target) before += sh.warp_m[s++];
        // the segment's sums, a part to a warp
        const int part = (a.seg / 32 + kWarps - 1) / kWarps * 32, b0 = s * a.seg + warp * part;
        const int end = min(w.n + w.shift, min(b0 + part, (s + 1) * a.seg));
        u64 mine = 0;
        for (int b = b0 + lane; b < end; b += 32) {
          const int i = b - w.shift;
          const float z = i >= 0 ? w.value(i) : -INFINITY;
          if (kept(i, z)) mine += weight(z, w.c, sh.table);
        }
        mine = warp_sum(mine);
        __syncthreads();
        if (lane == 0) sh.warp_m[warp] = mine;
        __syncthreads();
        for (int i = 0; i < warp; ++i) before += sh.warp_m[i];
        if (before < target && target <= before + mine) {  // (in one warp)
          for (int b = b0; b < end; b += 32) {
            const int i = b + lane - w.shift;
            const float z = b + lane < end && i >= 0 ? w.value(i) : -INFINITY;
            const u64 x = warp_scan(kept(i, z) ? weight(z, w.c, sh.table) : 0, lane);
            const unsigned hit = __ballot_sync(0xffffffffu, before + x >= target);
            if (hit) {
              if (lane == __ffs(hit) - 1) a.out_tokens[row] = w.begin + i;
              break;
            }
            before += __shfl_sync(0xffffffffu, x, 31);
          }
        }
      }
      // In place the draw must be through with what it reads from memory before any of it is written.
      if (a.out_logits == a.z && w.n + w.shift > a.cap) __syncthreads();
    }
    if (a.out_logits) {
      // (where f32 is too coarse for the difference, the next value below: rounded to the largest itself it would weigh 1)
      const float near = most - away;
      const float gone = fmaxf(most - near < 0.75f * away ? __fsub_rd(most, away) : near, -3.4028235e38f);
      float* to = a.out_logits + row * a.out_ld + w.begin;
      const bool wide = (reinterpret_cast<uintptr_t>(to - w.shift) & 15) == 0;  // (256 rows of 128256 338 us without, 314 with)
      w.each4([&](int i, float4 v) {
        float z[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = kept(i + e, z[e]) ? z[e] : gone;
        if (wide && i >= 0 && i + 4 <= w.n) {
          *reinterpret_cast<float4*>(to + i) = make_float4(z[0], z[1], z[2], z[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (static_cast<unsigned>(i + e) < static_cast<unsigned>(w.n)) to[i + e] = z[e];
        }
      });
    }
  }
  sv::cluster_sync();  // no CTA leaves while another may still read its shared memory
  if (tid == 0) {
    if (err && rank == 0) atomicOr(a.ctrl + sv::kKvCollect, err);
    if (sv::kv_last_cta(a.ctrl)) sv::kv_publish(a.ctrl);
  }
}

// --------------------------------------------------------------------- host
bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

bool dims_ok(const spec_sample_dims& d) {
  return d.rows >= 1 && d.rows <= (1 << 24) && d.V >= 1 && d.V <= (1 << 19) && d.ld >= d.V && d.ld <= (1ll << 36) &&
         d.out_ld >= d.V && d.out_ld <= (1ll << 36);
}

// CTAs to a row: a cluster of eight at most, 4096 tokens each at least.  A row takes as long as 12000 tokens (its barriers)
// and those of one CTA, and half as long again where two CTAs share an SM; clusters of three and more find room on about
// 11/12 of the SMs.  Rows with equal settings run in waves; such with settings of their own take very different times,
// which even out as far as they are many.  Measured (us): 40 rows of 128256 with top-p 68, 59, 80 and 78 with 3, 6, 7 and 8
// CTAs, 76 rows 95, 102 and 123 with 2, 3 and 4, 100 rows 143 and 126 with 2 and 4, 256 rows 267 and 270 with 1 and 4, but
// with settings of their own 267, 209, 198 and 226 with 1, 2, 4 and 8.
int ranks_for(int rows, int V, bool apart, int sms) {
  int best = 1;
  float least = INFINITY;
  for (int r = 1; r <= kMaxCluster && static_cast<int64_t>(V) > 4096ll * (r - 1); ++r) {
    const int room = r <= 2 ? 2 * sms : 2 * sms * 11 / 12, two = room / r, one = room / 2 / r;  // rows at once
    const int rest = rows % two;
    float waves;
    if (rows <= one) waves = 1.f;
    else if (rows <= two) waves = 1.47f;
    else if (apart) waves = 1.47f * (0.5f * rows / two + 0.6f);
    else waves = 1.47f * (rows / two) + (rest == 0 ? 0.f : rest <= one ? 1.f : 1.47f);
    const float cost = waves * (12000.f + static_cast<float>(V) / r);
    if (cost < least) {
      least = cost;
      best = r;
    }
  }
  return best;
}

}  // namespace

extern "C" {

size_t spec_sample_workspace_bytes(spec_sample_dims dims) { return dims_ok(dims) ? sv::kKvCtrlBytes : 0; }

spec_status spec_sample(const float* logits, const float* uniforms, const spec_sample_params* params,
                        int32_t* out_tokens, float* out_logits, spec_sample_dims dims, void* workspace,
                        size_t workspace_bytes, spec_stream_t stream) {
  if (!logits || !params || !workspace || (!out_tokens && !out_logits) || (out_tokens && !uniforms)) return SPEC_ERR_ARG;
  if (!params->temperatures && !(params->temperature >= 0.f && std::isfinite(params->temperature))) return SPEC_ERR_ARG;
  if ((!params->top_ps && std::isnan(params->top_p)) || (!params->min_ps && std::isnan(params->min_p))) return SPEC_ERR_ARG;
  if (!dims_ok(dims)) return SPEC_ERR_DIMS;
  if (out_logits == logits && dims.rows > 1 && dims.out_ld != dims.ld) return SPEC_ERR_ARG;
  if (misaligned(workspace, 16) || misaligned(logits, 4) || misaligned(uniforms, 4) || misaligned(out_tokens, 4) ||
      misaligned(out_logits, 4) || misaligned(params->temperatures, 4) || misaligned(params->top_ks, 4) ||
      misaligned(params->top_ps, 4) || misaligned(params->min_ps, 4))
    return SPEC_ERR_ALIGN;
  if (workspace_bytes < spec_sample_workspace_bytes(dims)) return SPEC_ERR_WORKSPACE;
  sv::DeviceInfo dev;
  const int st = sv::current_device(dev);
  if (st != SPEC_OK) return static_cast<spec_status>(st);
  SampleArgs a = {};
  a.z = logits;
  a.u = uniforms;
  a.par = *params;
  a.out_tokens = out_tokens;
  a.out_logits = out_logits;
  a.rows = dims.rows;
  a.V = dims.V;
  a.ld = dims.ld;
  a.out_ld = dims.out_ld;
  a.ctrl = static_cast<int*>(workspace);
  const bool apart = params->temperatures || params->top_ks || params->top_ps || params->min_ps;
  const int ranks = ranks_for(dims.rows, dims.V, apart, dev.sm_count);
  a.per = ((dims.V + ranks - 1) / ranks + 3) / 4 * 4;
  a.seg = (a.per + 3 + 128 * kWarps - 1) / (128 * kWarps) * 128;  // (up to three floats before the first)
  const int fixed = (sizeof(Shared) + 15) / 16 * 16 + static_cast<int>(sizeof(u64)) * bins_of(ranks);
  const int ring = kStages * kThreads * 16;
  a.cap = a.per + 4;
  int bytes = fixed + 4 * a.cap;
  if (bytes > kSharedBytes) {
    a.cap = (kSharedBytes - fixed - ring) / 4 / 128 * 128;
    bytes = fixed + 4 * a.cap + ring;
  }
  static bool done[64] = {false};
  if (!done[dev.device]) {
    if (cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes) != cudaSuccess)
      return SPEC_ERR_CUDA;
    done[dev.device] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(dims.rows) * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel, a) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_sample_read_error(void* workspace, int32_t* error_word, spec_stream_t stream) {
  if (!workspace || !error_word) return SPEC_ERR_ARG;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess ||
      cudaMemcpy(error_word, workspace, sizeof(int32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

}  // extern "C"
