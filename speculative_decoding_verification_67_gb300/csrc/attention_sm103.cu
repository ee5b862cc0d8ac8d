// Attention over the paged cache and over packed prompts.  Declared in
// include/spec_attention.h.
//
// One kernel for both.  A work item is a tile of query rows of one key-value
// head: row r of a tile is token r / G, head r % G of the group (G = heads /
// kv_heads), so a key or value is fetched once for all heads that share it.
// The item walks its keys in blocks of 128 with the running reference m and sum
// of the softmax:
//   S = Q K^T            tcgen05.mma, 128 x 128, operands in shared memory
//   P = exp2(S c - m c)  softmax warps, S read from and P written to TMEM
//   O = O + P V          tcgen05.mma, P from TMEM, V from shared memory
// with c = scale log2(e).  m is a maximum of the row; it is raised, and O
// rescaled, only when a later maximum exceeds it by more than 2^8 in weight.
// Until then weights up to 2^8 stand in P, which costs no precision and spares
// reading O back for most blocks.  P is rounded to the input type, because that
// is what the tensor core multiplies; the sum is of the unrounded weights.  fp16
// has few small exponents, so there every weight is taken 2^7 times as large (up
// to 2^15): those below 2^-21 of the reference's are off by 2^-32 of it, not those
// below 2^-14 by 2^-25, which many keys beside one large one would add up.
//
// Two softmax warpgroups (one row per thread) work on two score tiles, so the
// tensor core computes for one while the other is in its exponentials:
//   * prompts: two row tiles of the item share every K and V block;
//   * cache: the item has one row tile, the warpgroups take even and odd
//     blocks, each with a reference, sum and O of its own, merged at the end.
//     With few rows (one token: G of the 128 rows) the tensor core's work is
//     padding, but at 1024 clocks a block it stays below the ~2200 that a
//     block's 64 KB take from HBM.
// Tensor memory is full: two score tiles (P over the scores it came from) and
// two O.  So a tile's next scores wait for its last P V, and a tile's block takes
// the products' 1024 clocks and ~500 of their latency after the ~1900 of its
// softmax; two tiles overlap to ~3200 clocks per two blocks.  That chain
// bounds long prompts (69-72 % of the measured bf16 rate), HBM the cache form
// with a full batch, and start, end and join of the items everything short.
//
// One CTA per SM walks an equal share of all items' blocks (plus a constant per
// item for its start and end).  An item cut between CTAs leaves unnormalised
// partial rows, which a second, small kernel joins in the order of the pieces.
// Shares are computed from the lengths on the device; the host never sees them.
// Both kernels may start while what came before them on the stream ends, and
// wait for it before they touch memory.
//
// Loads: a ring of 128-position K and V tiles.  Packed keys are TMA boxes of 128
// token rows.  Over the cache whole blocks come as boxes of up to 128 rows of
// one page (every size divisible by 8), partial blocks, staged entries and
// other pages row by row with cp.async; rows behind the end are zeros.  Boxes
// of 16 rows and more stream B = 64 caches at 5.9 TB/s, boxes of eight at 5.5,
// rows at 3.7 (pages of 100 positions) and 2.8 (pages of one).
//
// Masked values: P is 0 where a row must not see a key, but 0 times an
// infinite or not-a-number value is not 0.  In blocks that some row may not
// see to the end, the softmax warps look through the V tile first: rows of V
// with such values are zeroed in shared memory and added, to the rows that do
// see them, by plain multiplications.
//
// Measured (GB300, calls one after the other): one prompt of 12301 tokens, 32
// heads over 8, 0.89-0.94 ms (1.33-1.40 PFLOP/s, the longer under the power
// limit at 1980 MHz); 16 prompts of up to 2047 tokens 237-241 us (0.77); 64
// caches of up to 8191 positions, one token each, 191-198 us; one cache of 1000
// positions 12 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "internal.h"
#include "kv_copy.cuh"
#include "sm103_ptx.cuh"
#include "spec_attention.h"

namespace {

constexpr int kBlock = 128;          // keys per block, rows per tile
constexpr int kThreads = 384;        // two softmax warpgroups, an MMA warp, three load warps
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kCopyWarps = 3;        // load warps of the cache form
constexpr int kMaxGrid = 160;        // CTAs (one per SM); sizes the workspace
// An item's start and end, in blocks (sets the shares): one 12301-token prompt took 950 us with 2, 915 with 3, 907
// with 4 and 921 with 6, 16 shorter ones 262, 251, 253 and 270; over the cache, where a block takes less, 2 did best.
template <bool kPaged>
constexpr int kItemUnits = kPaged ? 2 : 3;
constexpr int kMaxTree = 256;
constexpr int kJoinThreads = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;        // log2 of the largest weight before O is rescaled
constexpr float kFar = 1048576.f;    // |reference| from which weights are of scores less their maximum (see the kernel)

// a / b for non-negative values, in 32 bits where they fit (most do; the
// 64-bit division takes several hundred clocks).
__device__ __noinline__ long long quot_64(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long quot(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return quot_64(a, b);
}

// The units before CTA c's share: `q` each, the first `r` CTAs one more; none behind the total.
struct Shares {
  long long q, total;
  int r;
  // the CTA that has unit u
  __device__ __forceinline__ int owner(long long u) const {
    const long long wide = r * (q + 1);
    return static_cast<int>(u < wide ? quot(u, q + 1) : r + quot(u - wide, q));
  }
  __device__ __forceinline__ long long before(int c) const { return min(total, q * c + min(c, r)); }
};

// At least `least` units each: a piece of an item costs its rows' way through memory once more.
__device__ __forceinline__ Shares shares_of(long long total, int grid, int least) {
  if (total < static_cast<long long>(grid) * least) grid = max(1, static_cast<int>(total) / least);
  Shares s;
  s.total = total;
  s.q = quot(total, grid);
  s.r = static_cast<int>(total - s.q * grid);
  return s;
}

// What a join needs to know of an item that was cut (one record per CTA).
struct Cut {
  int active;
  int first;           // the CTA with its first piece
  int b, tokens;       // the sequence, the item's tokens
  long long row;       // the row of out of its first token's first head
  long long end;       // its last unit
  Shares shares;
};

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
  float scale_log2;
  int B, S, heads, kv_heads, G, page_size, num_pages, max_pages, total_q, total_k;
  int tile_tokens;        // whole tokens in a row tile
  int box;                // rows of one page box (a divisor of the page and of a block), or 0: row by row
  int least;              // units of the smallest share
  int join_split;         // CTAs that share the rows of one join
  long long k_stride, v_stride;
  // workspace
  int* ctrl;
  int* bad;               // [B] error bits of each sequence (cache)
  Cut* cuts;              // [kMaxGrid]
  float* part_o;          // [kMaxGrid][2][rows][D]
  float2* part_ml;        // [kMaxGrid][2][rows] (reference in log2, sum)
};

// Marks a sequence of the cache form (or, b < 0, the call) with error bits.
__device__ __forceinline__ void report(const AttnArgs& a, int b, int bits) {
  if (b >= 0) atomicOr(a.bad + b, bits);
  atomicOr(a.ctrl + sv::kKvCollect, bits);
}

// One sequence: Lq queries behind `base` keys (packed: negative when there are fewer keys than queries).
struct Seq {
  int Lq, base, q0, tiles;
  long long k0;
};

template <bool kPaged>
constexpr int kTiles = kPaged ? 1 : 2;

__device__ __forceinline__ int blocks_of(int keys) { return keys <= 0 ? 0 : (keys - 1) / kBlock + 1; }

template <bool kPaged>
__device__ Seq get_seq(const AttnArgs& a, int b, int& err) {
  Seq s;
  err = 0;
  if (kPaged) {
    const int L = a.len[b];
    const int n = a.len_k ? a.len_k[b] : a.S;
    s.Lq = n;
    s.base = L;
    s.q0 = b * a.S;
    s.k0 = 0;
    if (n < 0 || n > a.S || (L < 0 && n > 0)) err = SPEC_ATTN_DEVERR_LENGTH;
    else if (n > 0 && static_cast<long long>(L) + (a.staged ? 0 : n) >
                          static_cast<long long>(a.max_pages) * a.page_size)
      err = SPEC_ATTN_DEVERR_CAPACITY;
  } else {
    const int a0 = a.len[b], a1 = a.len[b + 1], b0 = a.len_k[b], b1 = a.len_k[b + 1];
    s.Lq = a1 - a0;
    s.base = (b1 - b0) - s.Lq;
    s.q0 = a0;
    s.k0 = b0;
    if (a0 < 0 || a1 < a0 || a1 > a.total_q || b0 < 0 || b1 < b0 || b1 > a.total_k) err = SPEC_ATTN_DEVERR_LENGTH;
  }
  if (err) s.Lq = 0;
  const int t = a.tile_tokens * kTiles<kPaged>;
  s.tiles = (s.Lq + t - 1) / t;
  return s;
}

// Blocks of an item: the keys its last token sees; one (of nothing) where none is seen.
template <bool kPaged>
__device__ __forceinline__ int item_blocks(const AttnArgs& a, const Seq& s, int tile) {
  if (kPaged) return a.staged ? blocks_of(s.base) + blocks_of(s.Lq) : blocks_of(s.base + s.Lq);
  const int t = a.tile_tokens * 2;
  const int n = blocks_of(s.base + min(s.Lq, (tile + 1) * t));
  return n > 0 ? n : 1;
}

// sum over i < n of floor((x i + y) / m), by the Euclidean recursion.
__device__ __noinline__ long long floor_sum(long long n, long long m, long long x, long long y) {
  long long sum = 0;
  while (n > 0) {
    if (x >= m) {
      const long long k = quot(x, m);
      sum += (n - 1) * n / 2 * k;
      x -= k * m;
    }
    if (y >= m) {
      const long long k = quot(y, m);
      sum += n * k;
      y -= k * m;
    }
    const long long top = x * n + y;
    if (top < m) break;
    n = quot(top, m);
    y = top - n * m;
    const long long t = m;
    m = x;
    x = t;
  }
  return sum;
}

// sum over i < n of floor((span i + y) / kBlock).  For spans that divide a block
// (groups of 2, 4, 8, ..) the terms repeat, for their multiples they rise evenly;
// the general recursion costs about ten divisions.
__device__ __forceinline__ long long step_sum(long long n, int span, int y) {
  if (kBlock % span == 0) {
    const int m = kBlock / span, shift = __ffs(m) - 1;
    auto upto = [&](long long t) {  // sum over i < t of floor(i / m)
      const long long q = t >> shift;
      return m * (q * (q - 1) / 2) + (t - (q << shift)) * q;
    };
    const long long from = y / span;
    return upto(from + n) - upto(from);
  }
  if (span % kBlock == 0) return n * (y / kBlock) + n * (n - 1) / 2 * (span / kBlock);
  return floor_sum(n, kBlock, span, y);
}

// Units (blocks and kItemUnits each) of the first t items of one head of a sequence.
template <bool kPaged>
__device__ __noinline__ long long head_units(const AttnArgs& a, const Seq s, int t) {
  long long sum = static_cast<long long>(t) * kItemUnits<kPaged>;
  if (kPaged) return sum + static_cast<long long>(t) * item_blocks<kPaged>(a, s, 0);
  const int span = a.tile_tokens * 2;
  const int full = t < s.tiles ? t : s.tiles - 1;  // tiles whose last token is (i + 1) span - 1
  int none = 0;                                    // tiles that see nothing: one block each
  if (s.base < 0) none = min(full, -s.base / span);
  // + sum over the others of ceil((base + (i + 1) span) / kBlock)
  sum += none + step_sum(full - none, span, s.base + (none + 1) * span + kBlock - 1);
  if (t == s.tiles) sum += item_blocks<kPaged>(a, s, t - 1);
  return sum;
}

// The item that has unit u, of sequence s whose units begin at `before`.
struct Place {
  int kvh, tile;
  long long start;  // the item's first unit
};

template <bool kPaged>
__device__ __noinline__ Place locate(const AttnArgs& a, const Seq s, long long units, long long before, long long u) {
  const long long per_head = quot(units, a.kv_heads), kvh = quot(u - before, per_head);
  const long long r = u - before - kvh * per_head;
  int lo = 0, hi = s.tiles;  // the last tile that starts at or before r
  if (kPaged) {
    lo = static_cast<int>(quot(r, item_blocks<kPaged>(a, s, 0) + kItemUnits<kPaged>));
  } else {
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (head_units<kPaged>(a, s, mid) <= r) lo = mid;
      else hi = mid;
    }
  }
  Place p;
  p.kvh = static_cast<int>(kvh);
  p.tile = lo;
  p.start = u - r + (lo ? head_units<kPaged>(a, s, lo) : 0);
  return p;
}

// A place in the list of items.
template <bool kPaged>
struct Cursor {
  int b, kvh, tile, n;
  long long start;  // first unit of the item
  Seq s;

  __device__ void next(const AttnArgs& a) {
    start += n + kItemUnits<kPaged>;
    if (++tile < s.tiles) {
      if (!kPaged) n = item_blocks<kPaged>(a, s, tile);
      return;
    }
    tile = 0;
    if (++kvh == a.kv_heads) {
      kvh = 0;
      do {
        if (++b >= a.B) return;  // behind the last item; start has reached the total
        int err;
        s = get_seq<kPaged>(a, b, err);
      } while (s.tiles == 0);
    }
    n = item_blocks<kPaged>(a, s, 0);
  }
};

template <int D, bool kPaged>
struct Shape {
  static constexpr int kTileBytes = kBlock * D * 2;
  static constexpr int kStages = D == 64 ? 8 : (kPaged ? 5 : 4);
  static constexpr int kQBytes = kTiles<kPaged> * kTileBytes;
  // Where 64 columns (128 bytes) of a row of a K or V tile lie: rows in groups of eight (the unit of the swizzle and
  // of the matrix descriptors).  Prompts: all rows of the first 64 columns, then of the others, as a box of token rows
  // brings them.  Cache: both halves of a group together, so that one box brings whole rows of a page.
  static constexpr int kGroup = kPaged ? D / 64 * 1024 : 1024;
  static constexpr int kHalf = kPaged ? 1024 : kBlock * 128;
  static __device__ __forceinline__ uint32_t spot(int row, int piece) {  // byte of a row's 16-byte piece
    return (row >> 3) * kGroup + (piece >> 3) * kHalf + (row & 7) * 128 + (((piece & 7) ^ (row & 7)) << 4);
  }
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kO = 256;  // O accumulators behind the two score tiles
};

struct Sync {
  uint64_t full[8], empty[8], q_full, q_empty, s_full[2], p_full[2], o_full[2], o_free[2], done;
  uint32_t tmem;
  int abort;
  int o_set[2];             // the softmax warps have written O themselves
  unsigned spoiled[2][2][4];
  Shares shares;
  int at_b, at_kvh, at_tile;
  long long at_start;
  Seq at_seq;
  long long scan[kThreads / 32];
};

struct Exchange {
  float ref[2][2][kBlock];        // [segment parity][tile][row]
  float sum[2][2][kBlock];
  uint4 rows[8][128];             // [softmax warp] 64 bytes of each of its rows, on their way out
};

struct TreeShared {
  unsigned anc[2][kBlock][9];     // [tile][row] ancestors of the row's node
};

// A wait that gives up after kWaitLimitNs, or as soon as another warp has.
// The CTA then runs on to its end without waiting (its results are void, the
// error word says so), so that no barrier is left with a warp missing.
__device__ __forceinline__ void await(Sync& sh, uint64_t* bar, uint32_t parity) {
  if (sv::mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = sv::global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (sv::mbar_try_wait(bar, parity)) return;
    if (*reinterpret_cast<volatile int*>(&sh.abort)) return;
    if (sv::global_timer_ns() - t0 > sv::kWaitLimitNs) *reinterpret_cast<volatile int*>(&sh.abort) = 1;
  }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ bool aborted(Sync& sh) { return *reinterpret_cast<volatile int*>(&sh.abort) != 0; }

// Named barriers of the softmax warps: 1 + t the 128 threads of a row tile,
// 3 those of both.
__device__ __forceinline__ void meet(int id, int threads) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// 16 bytes global -> shared, zeros where `bytes` is 0 (the address is not read then).
__device__ __forceinline__ void copy_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// One arrival on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sv::smem_u32(bar)) : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// x times its part's factor; 0 for a part that is left out (factor -1).
__device__ __forceinline__ float weighed(float x, float factor) { return factor < 0.f ? 0.f : x * factor; }

// Whether a packed pair holds an infinity or a NaN (all exponent bits set).
__device__ __forceinline__ bool odd_pair(uint32_t w, __nv_bfloat16) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ bool odd_pair(uint32_t w, __half) {
  return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
}

// Adds 0 to `sum` for two finite values, NaN for an infinity or a NaN.
__device__ __forceinline__ __nv_bfloat162 taint(uint32_t w, __nv_bfloat162 sum) {
  return __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(0.f), sum);
}
__device__ __forceinline__ __half2 taint(uint32_t w, __half2 sum) {
  return __hfma2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(0.f), sum);
}
__device__ __forceinline__ bool tainted(__nv_bfloat162 s) { return __hisnan(s.x) || __hisnan(s.y); }
__device__ __forceinline__ bool tainted(__half2 s) { return __hisnan(s.x) || __hisnan(s.y); }
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static __device__ __forceinline__ type zero() { return __float2bfloat162_rn(0.f); }
};
template <>
struct Pair<__half> {
  using type = __half2;
  static __device__ __forceinline__ type zero() { return __float2half2_rn(0.f); }
};

// Two products and sums in one instruction.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  uint64_t a, b, c, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x.x), "f"(x.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(y.x), "f"(y.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(z.x), "f"(z.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  uint64_t a, b, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x.x), "f"(x.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(y.x), "f"(y.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}

// kind::f16 instruction descriptor, f32 accumulators: A and B fp16 (0) or
// bf16 (1) at bits 7 and 10, B MN-major at bit 16.
template <typename T>
constexpr uint32_t idesc(uint32_t M, uint32_t N, uint32_t b_mn) {
  return (1u << 4) | (std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u) | (b_mn << 16) |
         ((N >> 3) << 17) | ((M >> 4) << 24);
}

// log2 of what stands in P for a score that equals the reference.
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 7.f : 0.f;

// The rank of V's load of block i among a segment's loads (cache order K0 K1 V0 K2 V1 ..).
template <bool kPaged>
__device__ __forceinline__ uint32_t v_rank(int i, int nb) {
  return kPaged ? (i + 1 < nb ? 2 * i + 2 : 2 * i + 1) : 2 * i + 1;
}

// Address of the value row of a position an item sees (the slow path).
template <typename T, int D, bool kPaged>
__device__ const T* value_row(const AttnArgs& a, const Seq& s, int b, int kvh, bool fresh, int pos) {
  if (!kPaged) return static_cast<const T*>(a.v) + (s.k0 + pos) * a.v_stride + kvh * D;
  const long long entry = 2ll * a.kv_heads * D;
  long long row;
  const T* base;
  if (fresh) {
    base = static_cast<const T*>(a.staged);
    row = static_cast<long long>(b) * a.S + pos;
  } else {
    base = static_cast<const T*>(a.k);
    const int page = a.bt[static_cast<long long>(b) * a.max_pages + pos / a.page_size];
    if (page < 0 || page >= a.num_pages) return nullptr;  // (flagged; its value is not used)
    row = static_cast<long long>(page) * a.page_size + pos % a.page_size;
  }
  return base + row * entry + static_cast<long long>(a.kv_heads + kvh) * D;
}

// Where the CTA's share begins, into shared memory.  (Functions of their own,
// so that what they need does not weigh on the registers of the loops.)
__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

template <bool kPaged>
__device__ __forceinline__ void begin_at(const AttnArgs& a, Sync& sh, const Seq s, int b, long long units,
                                         long long before, long long u) {
  const Place p = locate<kPaged>(a, s, units, before, u);
  sh.at_b = b;
  sh.at_kvh = p.kvh;
  sh.at_tile = p.tile;
  sh.at_start = p.start;
  sh.at_seq = s;
}

// Up to 32 sequences: one warp.
template <bool kPaged>
__device__ __noinline__ void scan_few(const AttnArgs& a, Sync& sh, int grid, int cta) {
  const int lane = threadIdx.x & 31;
  Seq s;
  s.tiles = 0;
  long long units = 0;
  if (lane < a.B) {
    int err;
    s = get_seq<kPaged>(a, lane, err);
    if (s.tiles > 0) units = head_units<kPaged>(a, s, s.tiles) * a.kv_heads;
    if (err && cta == 0) report(a, kPaged ? lane : -1, err);
  }
  const long long x = warp_scan(units, lane);
  const Shares shares = shares_of(__shfl_sync(0xffffffffu, x, 31), grid, a.least);
  const long long u = shares.before(cta);
  if (lane == 0) sh.shares = shares;
  if (units > 0 && x - units <= u && u < x) begin_at<kPaged>(a, sh, s, lane, units, x - units, u);
}

// More: the whole CTA, in two passes where a thread has more than one sequence.
template <bool kPaged>
__device__ __noinline__ void scan_many(const AttnArgs& a, Sync& sh, int grid, int cta) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  long long total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    long long seen = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
      const int b = b0 + tid;
      long long units = 0;
      Seq s;
      s.tiles = 0;
      if (b < a.B) {
        int err;
        s = get_seq<kPaged>(a, b, err);
        if (s.tiles > 0) units = head_units<kPaged>(a, s, s.tiles) * a.kv_heads;
        if (err && pass == 0 && cta == 0) report(a, kPaged ? b : -1, err);
      }
      const long long x = warp_scan(units, lane);
      __syncthreads();
      if (lane == 31) sh.scan[warp] = x;
      __syncthreads();
      long long before = seen, sum = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sh.scan[w];
        sum += sh.scan[w];
      }
      before += x - units;
      seen += sum;
      if (pass == 0 && b0 + kThreads < a.B) continue;  // the total is not known yet
      if (pass == 0) total = seen;
      if (pass == 0 && a.B > kThreads) break;          // find the start in a second pass
      const long long u = shares_of(total, grid, a.least).before(cta);
      if (units > 0 && before <= u && u < before + units) begin_at<kPaged>(a, sh, s, b, units, before, u);
    }
    if (a.B <= kThreads) break;
  }
  if (tid == 0) sh.shares = shares_of(total, grid, a.least);
}

template <typename T, int D, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v) {
  // (cache: map_k is the pool's; map_v is not used)
  using Sh = Shape<D, kPaged>;
  constexpr int kNT = kTiles<kPaged>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* q_tile = smem;
  uint8_t* ring = smem + Sh::kQBytes;
  uint8_t* tail = ring + Sh::kStages * Sh::kTileBytes;
  Sync& sh = *reinterpret_cast<Sync*>(tail);
  Exchange& ex = *reinterpret_cast<Exchange*>(tail + (sizeof(Sync) + 15) / 16 * 16);
  TreeShared& ts = *reinterpret_cast<TreeShared*>(&ex + 1);  // (cache only)
  // (the shuffle tells the compiler that the warp index is the same in all lanes)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int cta = blockIdx.x;
  const int grid = gridDim.x;

  if (tid == 0) {
    for (int i = 0; i < 8; ++i) {
      sv::mbar_init(&sh.full[i], kPaged ? 32 * kCopyWarps : 1);
      sv::mbar_init(&sh.empty[i], 1);
    }
    sv::mbar_init(&sh.q_full, 1);
    sv::mbar_init(&sh.q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      sv::mbar_init(&sh.s_full[t], 1);
      sv::mbar_init(&sh.p_full[t], 4);
      sv::mbar_init(&sh.o_full[t], 1);
      sv::mbar_init(&sh.o_free[t], kPaged ? 8 : 4);
    }
    sv::mbar_init(&sh.done, 1);
    sv::fence_barrier_init();
    sh.abort = 0;
  }
  if (warp == kMmaWarp) {
    sv::tmem_alloc(&sh.tmem, Sh::kTmemCols);
    sv::tmem_relinquish_alloc_permit();
  }
  if (warp == kLoadWarp && lane == 0) {
    sv::prefetch_tensor_map(&map_q);
    sv::prefetch_tensor_map(&map_k);
    if (!kPaged) sv::prefetch_tensor_map(&map_v);
  }

  // up to here nothing of the caller's was touched: what came before on the stream may still run
  sv::griddep_wait();
  sv::griddep_launch_dependents();
  if (tid == 0) a.cuts[cta].active = 0;

  // ---- this CTA's share of the units: a scan over the sequences
  if (a.B > 32) scan_many<kPaged>(a, sh, grid, cta);
  else if (warp == 0) scan_few<kPaged>(a, sh, grid, cta);
  if (kPaged && a.parents) {  // trees are checked once per sequence
    for (int b = cta; b < a.B; b += gridDim.x) {
      int err;
      const Seq s = get_seq<kPaged>(a, b, err);
      for (int i = tid; i < s.Lq; i += kThreads) {
        const int p = a.parents[static_cast<long long>(b) * a.S + i];
        if (i == 0 ? p != -1 : (p < 0 || p >= i)) report(a, b, SPEC_ATTN_DEVERR_TREE);
      }
    }
  }
  sv::tc_fence_before_sync();
  __syncthreads();
  sv::tc_fence_after_sync();
  const uint32_t tmem = sh.tmem;
  const long long u0 = sh.shares.before(cta), u1 = sh.shares.before(cta + 1);
  Cursor<kPaged> at = {};
  at.start = u1;  // no share: nothing to walk
  if (u0 < u1) {
    at.b = sh.at_b;
    at.kvh = sh.at_kvh;
    at.tile = sh.at_tile;
    at.start = sh.at_start;
    at.s = sh.at_seq;
    at.n = item_blocks<kPaged>(a, at.s, at.tile);
  }

  if (warp >= kLoadWarp) {
    // ------------------------------------------------------------- loads
    uint32_t loads = 0, segs = 0;
    const uint64_t keep = sv::l2_policy_evict_normal(), once = sv::l2_policy_evict_first();
    const int lw = warp - kLoadWarp;
    const bool issuer = elect_one();
    const uint64_t policy = a.S * a.G <= kBlock ? once : keep;  // whether another row tile reads the entries again
    auto load_q = [&]() {  // by one thread
      if (segs > 0) await(sh, &sh.q_empty, (segs - 1) & 1);
      if (aborted(sh)) return;
      const int tok = at.s.q0 + at.tile * a.tile_tokens * kNT;
      sv::mbar_arrive_expect_tx(&sh.q_full, kNT * a.tile_tokens * a.G * D * 2);
      for (int t = 0; t < kNT; ++t)
        for (int h = 0; h < D / 64; ++h)
          sv::tma_load_3d(q_tile + t * Sh::kTileBytes + h * (kBlock * 128), &map_q, &sh.q_full, h * 64, at.kvh * a.G,
                          tok + t * a.tile_tokens, once);
    };
    if (lw < (kPaged ? kCopyWarps : 1)) {
      for (; at.start < u1; at.next(a)) {
        const int lo = static_cast<int>(max(0ll, u0 - at.start - kItemUnits<kPaged>));
        const int hi = static_cast<int>(min(static_cast<long long>(at.n), u1 - at.start - kItemUnits<kPaged>));
        if (hi <= lo) continue;
        if (kPaged) {
          const int committed = a.staged ? blocks_of(at.s.base) : at.n;  // blocks read from the pool
          const int limit = a.staged ? at.s.base : at.s.base + at.s.Lq;
          const int* table = a.bt + static_cast<long long>(at.b) * a.max_pages;
          const unsigned long long entry = 4ull * a.kv_heads * D;  // bytes
          constexpr int kEach = kBlock / 32;             // rows a lane looks up: lane, lane + 32, ..
          constexpr int kChunks = D / 8;                 // 16-byte pieces of a row
          constexpr int kAtOnce = 32 / kChunks;          // rows one instruction copies
          const int chunk = lane % kChunks, sub = lane / kChunks;
          int r0[kEach], r1[kEach] = {};  // rows of the block before, of this block; -1: zeros
          // whole blocks of the pool come in boxes of a.box rows of one page, the others row by row
          auto boxed = [&](int j) { return a.box != 0 && j < committed && limit - j * kBlock >= kBlock; };
          auto row_at = [&](int p) {  // the pool's row of a position
            const int col = p / a.page_size, page = table[col];
            if (page >= 0 && page < a.num_pages) return page * a.page_size + (p - col * a.page_size);
            report(a, at.b, SPEC_ATTN_DEVERR_PAGE);
            return -1;
          };
          auto rows_of = [&](int j, int (&r)[kEach]) {
            if (boxed(j)) {  // lane i: first row of box i
              r[0] = lane * a.box < kBlock ? row_at(j * kBlock + lane * a.box) : 0;
              if (r[0] < 0) r[0] = a.num_pages * a.page_size;  // (outside the tensor: zeros)
              return;
            }
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
              const int in = 32 * e + lane;
              r[e] = -1;
              if (j >= committed) {
                const int i = (j - committed) * kBlock + in;
                if (i < at.s.Lq) r[e] = at.b * a.S + i;
              } else if (j * kBlock + in < limit) {
                r[e] = row_at(j * kBlock + in);
              }
            }
          };
          auto copy = [&](int j, const int (&r)[kEach], int head) {
            const uint32_t slot = loads % Sh::kStages;
            await(sh, &sh.empty[slot], (loads / Sh::kStages & 1) ^ 1);
            ++loads;
            if (__any_sync(0xffffffffu, aborted(sh))) return;
            if (boxed(j)) {
              const int boxes = kBlock / a.box;
              uint8_t* dst = ring + slot * Sh::kTileBytes;
              const int mine = boxes > lw ? (boxes - lw + kCopyWarps - 1) / kCopyWarps : 0;  // boxes lw, lw + 3, ..
              if (issuer) {
                if (mine > 0) sv::mbar_arrive_expect_tx(&sh.full[slot], mine * a.box * D * 2);
                else sv::mbar_arrive(&sh.full[slot]);
              } else {
                sv::mbar_arrive(&sh.full[slot]);
              }
              __syncwarp();
              for (int i = lw; i < boxes; i += kCopyWarps) {
                const int row = __shfl_sync(0xffffffffu, r[0], i);
                if (issuer)
                  sv::tma_load_4d(dst + i * a.box / 8 * Sh::kGroup, &map_k, &sh.full[slot], 0, 0, head * (D / 64),
                                  row / 8, policy);
                __syncwarp();
              }
              return;
            }
            const char* from = static_cast<const char*>(j >= committed ? a.staged : a.k) + head * (D * 2) + chunk * 16;
            const uint32_t to = sv::smem_u32(ring + slot * Sh::kTileBytes);
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
#pragma unroll
              for (int k = 0; k < (32 / kAtOnce + kCopyWarps - 1) / kCopyWarps; ++k) {
                const int i = k * kCopyWarps + lw;
                const int in = i * kAtOnce + sub, spot = 32 * e + in;
                const int row = __shfl_sync(0xffffffffu, r[e], in & 31);
                if (i < 32 / kAtOnce)
                  copy_16(to + Sh::spot(spot, chunk), from + static_cast<unsigned>(max(row, 0)) * entry,
                      row < 0 ? 0 : 16);
              }
            }
            copies_arrive(&sh.full[slot]);
          };
          if (segs == 0 && lw == 0 && lane == 0) load_q();  // (later ones wait for the last item's products)
          __syncwarp();
          rows_of(lo, r0);
          copy(lo, r0, at.kvh);
          if (segs > 0 && lw == 0 && lane == 0) load_q();
          __syncwarp();
          for (int j = lo; j < hi; ++j) {
            if (j + 1 < hi) {
              rows_of(j + 1, r1);
              copy(j + 1, r1, at.kvh);
            }
            copy(j, r0, a.kv_heads + at.kvh);
#pragma unroll
            for (int e = 0; e < kEach; ++e) r0[e] = r1[e];
          }
        } else if (lane == 0) {
          for (int j = lo; j < hi; ++j) {
            for (int kv = 0; kv < 2; ++kv) {
              const uint32_t slot = loads % Sh::kStages;
              await(sh, &sh.empty[slot], (loads / Sh::kStages & 1) ^ 1);
              if (!aborted(sh)) {
                sv::mbar_arrive_expect_tx(&sh.full[slot], Sh::kTileBytes);
                for (int h = 0; h < D / 64; ++h)
                  sv::tma_load_3d(ring + slot * Sh::kTileBytes + h * Sh::kHalf, kv ? &map_v : &map_k,
                                  &sh.full[slot], h * 64, at.kvh, static_cast<int>(at.s.k0) + j * kBlock, keep);
              }
              ++loads;
              if (j == lo && kv == 0) load_q();
            }
          }
        }
        ++segs;
      }
      if (kPaged) {
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
      if (aborted(sh) && lane == 0) {  // leave no copy in flight
        const uint32_t last = loads > Sh::kStages ? loads - Sh::kStages : 0;
        for (uint32_t i = last; i < loads; ++i) sv::mbar_wait(&sh.full[i % Sh::kStages], i / Sh::kStages & 1);
        if (lw == 0 && segs > 0) sv::mbar_wait(&sh.q_full, (segs - 1) & 1);
      }
      __syncwarp();
    }
  } else if (warp == kMmaWarp) {
    // --------------------------------------------------------------- MMA
    // All lanes walk the loop, so that addresses stay in uniform registers; one issues.
    {
      const bool issuer = elect_one();
      uint32_t loads = 0, segs = 0, p_cnt[2] = {0, 0}, used[2] = {0, 0};
      constexpr uint32_t kIdS = idesc<T>(kBlock, kBlock, 0), kIdO = idesc<T>(kBlock, D, 1);
      const uint32_t ring_addr = sv::smem_u32(ring), q_addr = sv::smem_u32(q_tile);
      auto arrived = [&]() -> uint32_t {  // waits for the next load; its address
        const uint32_t slot = loads % Sh::kStages;
        await(sh, &sh.full[slot], loads / Sh::kStages & 1);
        if (kPaged) sv::fence_proxy_async_smem();  // the copies wrote through the generic proxy
        sv::tc_fence_after_sync();
        return ring_addr + slot * Sh::kTileBytes;
      };
      auto commit = [&](uint64_t* bar) {
        if (issuer) sv::mma_commit(bar);
        __syncwarp();
      };
      auto scores = [&](int t, uint32_t k_addr) {
        const uint32_t qa = __shfl_sync(0xffffffffu, q_addr + (kPaged ? 0 : t * Sh::kTileBytes), 0);
        const uint32_t ka = __shfl_sync(0xffffffffu, k_addr, 0), d = __shfl_sync(0xffffffffu, tmem + t * kBlock, 0);
        const uint64_t q_desc = sv::smem_desc_k_sw128(qa), k_desc = sv::smem_desc_k_sw128(ka, Sh::kGroup);
        if (issuer) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t in = (k % 4) * 32;
            sv::mma_bf16_ss(d, q_desc + (((k / 4) * (kBlock * 128) + in) >> 4),
                            k_desc + (((k / 4) * Sh::kHalf + in) >> 4), kIdS, k > 0);
          }
          sv::mma_commit(&sh.s_full[t]);
        }
        __syncwarp();
      };
      // P V of one block; waits for P and, first, for O to be free
      auto values = [&](int t, uint32_t v_addr, bool first) {
        if (first && used[t] > 0) await(sh, &sh.o_free[t], (used[t] - 1) & 1);
        await(sh, &sh.p_full[t], p_cnt[t] & 1);
        ++p_cnt[t];
        sv::tc_fence_after_sync();
        const uint32_t fresh = first && !*reinterpret_cast<volatile int*>(&sh.o_set[t]);
        const uint32_t va = __shfl_sync(0xffffffffu, v_addr, 0), p = __shfl_sync(0xffffffffu, tmem + t * kBlock, 0);
        const uint64_t v_desc = sv::smem_desc_mn_sw128(va, Sh::kHalf, Sh::kGroup);
        const uint32_t go = __shfl_sync(0xffffffffu, fresh ^ 1u, 0), d = p - t * kBlock + Sh::kO + t * D;
        if (issuer) {
#pragma unroll
          for (int k = 0; k < kBlock / 16; ++k)
            sv::mma_f16_ts(d, p + k * 8, v_desc + k * (2 * Sh::kGroup >> 4), kIdO, k > 0 ? 1u : go);
        }
        __syncwarp();
      };
      for (; at.start < u1; at.next(a)) {
        const int lo = static_cast<int>(max(0ll, u0 - at.start - kItemUnits<kPaged>));
        const int hi = static_cast<int>(min(static_cast<long long>(at.n), u1 - at.start - kItemUnits<kPaged>));
        const int nb = hi - lo;
        if (nb <= 0) continue;
        await(sh, &sh.q_full, segs & 1);
        if (kPaged) {
          for (int i = 0; i < 2 && i < nb; ++i) {
            const uint32_t k_addr = arrived();
            scores(i, k_addr);
            commit(&sh.empty[loads++ % Sh::kStages]);
          }
          if (nb <= 2) commit(&sh.q_empty);
          for (int i = 0; i < nb; ++i) {
            const int t = i & 1;
            const uint32_t v_addr = arrived();
            values(t, v_addr, i < 2);
            commit(&sh.empty[loads++ % Sh::kStages]);
            if (i + 2 >= nb) commit(&sh.o_full[t]);
            if (i + 2 < nb) {
              const uint32_t k_addr = arrived();
              scores(t, k_addr);
              commit(&sh.empty[loads++ % Sh::kStages]);
              if (i + 3 == nb) commit(&sh.q_empty);
            }
          }
          ++used[0];
          if (nb > 1) ++used[1];
        } else {
          const bool two = at.s.Lq - at.tile * a.tile_tokens * 2 > a.tile_tokens;
          uint32_t k_addr = arrived();
          scores(0, k_addr);
          if (two) scores(1, k_addr);
          commit(&sh.empty[loads++ % Sh::kStages]);
          if (nb == 1) commit(&sh.q_empty);
          for (int i = 0; i < nb; ++i) {
            const uint32_t v_addr = arrived(), v_slot = loads++ % Sh::kStages;
            values(0, v_addr, i == 0);
            if (i + 1 == nb) commit(&sh.o_full[0]);
            uint32_t k_slot = 0;
            if (i + 1 < nb) {
              k_addr = arrived();
              k_slot = loads++ % Sh::kStages;
              scores(0, k_addr);
            }
            if (two) values(1, v_addr, i == 0);
            commit(&sh.empty[v_slot]);
            if (two && i + 1 == nb) commit(&sh.o_full[1]);
            if (i + 1 < nb) {
              if (two) scores(1, k_addr);
              commit(&sh.empty[k_slot]);
              if (i + 2 == nb) commit(&sh.q_empty);
            }
          }
          ++used[0];
          if (two) ++used[1];
        }
        ++segs;
      }
      if (aborted(sh)) {  // the products in flight end before the tensor memory is given back
        commit(&sh.done);
        sv::mbar_wait(&sh.done, 0);
      }
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- softmax
    const int t = warp >> 2, row = tid & (kBlock - 1);             // one row of one tile per thread
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const uint32_t s_addr = tmem + t * kBlock + lanes;
    const uint32_t o_addr = tmem + Sh::kO + t * D + lanes;
    const float c2 = a.scale_log2;
    uint32_t loads = 0, s_cnt = 0, used[2] = {0, 0}, merges = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      await(sh, bar, parity);
      __syncwarp();
    };
    for (; at.start < u1; at.next(a)) {
      const int lo = static_cast<int>(max(0ll, u0 - at.start - kItemUnits<kPaged>));
      const int hi = static_cast<int>(min(static_cast<long long>(at.n), u1 - at.start - kItemUnits<kPaged>));
      const int nb = hi - lo;
      if (nb <= 0) continue;
      const Seq& s = at.s;
      const int item_tok = at.tile * a.tile_tokens * kNT;
      const int tok0 = item_tok + (kPaged ? 0 : t * a.tile_tokens);
      const int rows = max(0, min(a.tile_tokens, s.Lq - tok0)) * a.G;
      const bool both = kPaged ? nb > 1 : s.Lq - item_tok > a.tile_tokens;  // the second score tile is in use
      if (tid == 0 && lo > 0) {
        Cut cut;
        cut.first = cta - 1;  // (every CTA before one with a share has one)
        cut.active = sh.shares.before(cta - 1) - at.start - kItemUnits<kPaged> <= 0;
        cut.end = at.start + kItemUnits<kPaged> + at.n - 1;
        cut.shares = sh.shares;
        cut.b = at.b;
        cut.tokens = min(a.tile_tokens * kNT, s.Lq - item_tok);
        cut.row = (static_cast<long long>(s.q0) + item_tok) * a.heads + at.kvh * a.G;
        a.cuts[cta] = cut;
      }
      if (t == 1 && !both) {
        // (Prompts: the tile's next wait for a V tile is by parity, so it must not be an item's loads behind.)
        if (!kPaged) wait(&sh.o_full[0], used[0] & 1);
        loads += 2 * nb;
        ++used[0];
        ++merges;
        continue;
      }
      const bool alive = (row & ~31) < rows;  // the warp has a row
      const int i_tok = tok0 + row / a.G;     // this row's token
      const int committed = kPaged && a.staged ? blocks_of(s.base) : at.n;
      const bool tree = kPaged && a.parents != nullptr;
      if (tree) {  // (a node's depth in dependent loads: 256 nodes in a line take 37 us where a chain of 256 takes 22)
        if (alive) {
          unsigned* anc = ts.anc[t][row];
#pragma unroll
          for (int w = 0; w < 8; ++w) anc[w] = 0;
          int p = min(i_tok, s.Lq - 1);
          while (p >= 0) {
            anc[p >> 5] |= 1u << (p & 31);
            const int up = a.parents[static_cast<long long>(at.b) * a.S + p];
            p = up < p ? up : -1;  // (a bad parent is flagged; the walk still ends)
          }
        }
      }
      float top = -INFINITY, sum = 0.f;  // the row's reference as a score, the sum of its weights
      float limit = -INFINITY;           // a block's maximum beyond it raises the reference; -infinity without one, or far

      for (int i = kPaged ? t : 0; i < nb; i += kPaged ? 2 : 1) {
        const bool first = i < (kPaged ? 2 : 1);
        const int j = lo + i;
        // the block's first position (fresh: index among the new entries), how far this row and the item's first
        // row see into it
        const bool fresh = j >= committed;
        const int pos0 = (fresh ? j - committed : j) * kBlock;
        int seen, least;
        if (kPaged && a.staged) {
          seen = fresh ? i_tok + 1 - pos0 : s.base - pos0;
          least = fresh ? (tree ? 0 : item_tok + 1 - pos0) : s.base - pos0;
        } else {
          seen = s.base + i_tok + 1 - pos0;
          least = s.base + (tree ? 0 : item_tok + 1) - pos0;
        }
        const bool masked = least < kBlock;
        const bool look = masked && (!kPaged || (s.Lq > 1 && (fresh || !a.staged)));
        auto scored = [&]() {
          wait(&sh.s_full[t], s_cnt & 1);
          ++s_cnt;
          sv::tc_fence_after_sync();
        };
        unsigned spoil[4] = {0, 0, 0, 0};
        // Prompts look while the scores are on their way.  (The load before V's in its slot has landed: this tile's last
        // products or scores needed it, or the last products of an item that it passed over, for which it waited.
        // Over the cache it may be the other tile's next K, which has landed for sure only with the scores.)
        if (kPaged) scored();
        if (look) {
          // one row of the V tile per thread; where both tiles read it, each half of the row
          const bool pair = !kPaged && both;
          const int parts = pair ? 2 : 1, part = pair ? t : 0, box = pair ? 0 : t;
          const int bar = pair ? 3 : 1 + t, crowd = pair ? 256 : 128;
          const uint32_t rank = loads + v_rank<kPaged>(i, nb), slot = rank % Sh::kStages;
          wait(&sh.full[slot], rank / Sh::kStages & 1);
          uint8_t* tile = ring + slot * Sh::kTileBytes;
          const int chunks = D / 8 / parts, c0 = part * chunks;
          // By bits over the cache, by multiplications for prompts.  Over the cache 64 sequences took 193 us
          // with the bits, 203 with the multiplications (197 unrolled by 8).  Unrolled loops spill in the
          // prompts' kernel: 16 prompts took 242 us with the bits, 235 with the multiplications.
          bool odd = false;
          if constexpr (kPaged) {
            for (int c = c0; c < c0 + chunks; ++c) {
              const uint4 w = *reinterpret_cast<const uint4*>(tile + Sh::spot(row, c));
              odd |= odd_pair(w.x, T()) || odd_pair(w.y, T()) || odd_pair(w.z, T()) || odd_pair(w.w, T());
            }
          } else {
            typename Pair<T>::type sum0 = Pair<T>::zero(), sum1 = sum0;
#pragma unroll 1
            for (int c = c0; c < c0 + chunks; ++c) {
              const uint4 w = *reinterpret_cast<const uint4*>(tile + Sh::spot(row, c));
              sum0 = taint(w.x, taint(w.y, sum0));
              sum1 = taint(w.z, taint(w.w, sum1));
            }
            odd = tainted(sum0) || tainted(sum1);
          }
          const unsigned word = __ballot_sync(0xffffffffu, odd);
          if (lane == 0) sh.spoiled[box][part][warp & 3] = word;
          meet(bar, crowd);
#pragma unroll
          for (int w = 0; w < 4; ++w)
            for (int k = 0; k < parts; ++k) spoil[w] |= *reinterpret_cast<volatile unsigned*>(&sh.spoiled[box][k][w]);
          const unsigned own =
              (warp & 2) ? ((warp & 1) ? spoil[3] : spoil[2]) : ((warp & 1) ? spoil[1] : spoil[0]);
          if (own >> lane & 1u) {
            for (int c = c0; c < c0 + chunks; ++c)
              *reinterpret_cast<uint4*>(tile + Sh::spot(row, c)) = make_uint4(0, 0, 0, 0);
            sv::fence_proxy_async_smem();
          }
          meet(bar, crowd);
          if (!kPaged) {  // keys behind the sequence's are other sequences': zeroed, not added
            const int keys = s.base + s.Lq - pos0;
#pragma unroll
            for (int w = 0; w < 4; ++w)
              spoil[w] &= keys >= 32 * (w + 1) ? 0xffffffffu : (keys <= 32 * w ? 0u : (1u << (keys - 32 * w)) - 1u);
          }
        }
        if (!kPaged) scored();
        const bool spoils = (spoil[0] | spoil[1] | spoil[2] | spoil[3]) != 0;
        if (first && row == 0) *reinterpret_cast<volatile int*>(&sh.o_set[t]) = spoils;
        // bit c of word w: column 32 w + c is seen
        auto seen_word = [&](int w) -> unsigned {
          if (tree && (fresh || !a.staged)) {
            // bits idx0 .. idx0 + 31 of the ancestors; everything before the new entries is seen
            const unsigned* anc = ts.anc[t][row];
            const int idx0 = pos0 + 32 * w - (a.staged ? 0 : s.base), k = idx0 >> 5;
            const unsigned b0 = k < 0 ? 0xffffffffu : (k < 8 ? anc[k] : 0u);
            const unsigned b1 = k + 1 < 0 ? 0xffffffffu : (k + 1 < 8 ? anc[k + 1] : 0u);
            return __funnelshift_r(b0, b1, idx0 & 31);
          }
          return seen >= 32 * (w + 1) ? 0xffffffffu : (seen <= 32 * w ? 0u : (1u << (seen - 32 * w)) - 1u);
        };
        // 32 scores as they arrive, -infinity where the row must not see the key
        auto hide = [&](int h, uint32_t (&x)[32]) {
          sv::tmem_arrived_32(x);
          if (!masked) return;
          const unsigned m = seen_word(h);
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!(m >> c & 1u)) x[c] = 0xff800000u;
        };
        if (alive) {
          // Two passes over the scores, each with the next 32 columns on their way while the last ones are worked on:
          // their maximum, then their weights, written over scores read before.
          uint32_t x[2][32];
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          sv::tmem_start_32(s_addr, x[0]);
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t(&now)[32] = x[h & 1];
            hide(h, now);
            sv::tmem_start_32(s_addr + 32 * ((h + 1) & 3), x[(h + 1) & 1]);
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              mx[c / 2 & 3] = fmaxf(mx[c / 2 & 3], fmaxf(__uint_as_float(now[c]), __uint_as_float(now[c + 1])));
          }
          const float blk = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // raise the reference where a weight would exceed 2^kSlack (rows that the tile does not have hold what lay in
          // their place before, and send no warp this way)
          if (__any_sync(0xffffffffu, blk > limit && row < rows) || spoils) {
            sv::tmem_arrived_32(x[0]);  // its registers are free from here on
            float f = 1.f;
            if (blk > limit && blk > top) {
              f = top == -INFINITY ? 0.f : exp2_approx(fmaf(top, c2, -kLift<T>) - fmaf(blk, c2, -kLift<T>));
              top = blk;
              limit = fabsf(top * c2) > kFar ? -INFINITY : top + kSlack / c2;
            }
            if (!first) {
              sum *= f;
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float o[32];
                sv::tmem_load_32(o_addr + c, o);
                uint32_t u[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * f);
                sv::tmem_store_32(o_addr + c, u);
              }
              sv::tmem_wait_st();
            }
            const bool far = limit == -INFINITY && top != -INFINITY;
            const float less = far ? top : 0.f;
            if (spoils) {  // rare: values that are infinite or not a number, for the rows that see them
              if (first) {
                if (used[t] > 0) wait(&sh.o_free[t], (used[t] - 1) & 1);
                sv::tc_fence_after_sync();
                uint32_t u[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) u[e] = 0;
                for (int c = 0; c < D; c += 32) sv::tmem_store_32(o_addr + c, u);
                sv::tmem_wait_st();
              }
#pragma unroll 1
              for (int c = 0; c < kBlock; ++c) {
                const unsigned sw = c < 64 ? (c < 32 ? spoil[0] : spoil[1]) : (c < 96 ? spoil[2] : spoil[3]);
                if (!(sw >> (c & 31) & 1u)) continue;
                const bool mine = seen_word(c >> 5) >> (c & 31) & 1u;
                const float off2 = limit == -INFINITY ? kLift<T> : fmaf(-top, c2, kLift<T>);
                const float p = exp2_approx(fmaf(sv::tmem_load_1(s_addr + c) - less, c2, off2));
                const T* v = value_row<T, D, kPaged>(a, s, at.b, at.kvh, kPaged && a.staged && fresh, pos0 + c);
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                  float o[32];
                  sv::tmem_load_32(o_addr + d, o);
                  uint32_t u[32];
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    u[e] = __float_as_uint(mine && v != nullptr ? o[e] + p * to_f(v[d + e]) : o[e]);
                  sv::tmem_store_32(o_addr + d, u);
                  sv::tmem_wait_st();
                }
              }
            }
            // Far: top * c2 is rounded to a reference up to 2^-24 of it away, an exponent that from 2^27 on takes weights
            // out of fp16's range and from 2^31 on out of bf16's.  The second pass then finds the scores less top (exact
            // for scores near it) and subtracts nothing.  Every block of such a row comes here, by its limit: a test
            // beside the limit's cost long prompts 2 %, this one nothing (888-896 us).
            if (__any_sync(0xffffffffu, far)) {
#pragma unroll 1
              for (int c = 0; c < kBlock; c += 32) {
                float z[32];
                sv::tmem_load_32(s_addr + c, z);
                uint32_t u[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(z[e] - less);
                sv::tmem_store_32(s_addr + c, u);
              }
              sv::tmem_wait_st();
            }
            sv::tmem_start_32(s_addr, x[0]);
          }
          const float add = limit == -INFINITY ? kLift<T> : fmaf(-top, c2, kLift<T>);  // minus the reference
          const float2 cc = make_float2(c2, c2), oo = make_float2(add, add);
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t(&now)[32] = x[h & 1];
            hide(h, now);
            if (h < 3) sv::tmem_start_32(s_addr + 32 * (h + 1), x[(h + 1) & 1]);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 z = fma2(make_float2(__uint_as_float(now[2 * e]), __uint_as_float(now[2 * e + 1])), cc, oo);
              z.x = exp2_approx(z.x);
              z.y = exp2_approx(z.y);
              acc[e & 1] = add2(acc[e & 1], z);
              w[e] = pack2(z.x, z.y, T());
            }
            sv::tmem_store_16(s_addr + 16 * h, w);
          }
          const float2 both_acc = add2(acc[0], acc[1]);
          sum += both_acc.x + both_acc.y;
          sv::tmem_wait_st();
        }
        sv::tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) sv::mbar_arrive(&sh.p_full[t]);
      }
      loads += 2 * nb;

      // ---- end of the segment: normalise and write, or leave partial rows
      const bool whole = lo == 0 && hi == at.n;
      const long long slot = (static_cast<long long>(cta) * 2 + (lo > 0 ? 0 : 1)) * (kNT * kBlock);
      const uint32_t par = merges++ & 1;
      // in the cache form with both tiles in use each has half of the rows' columns
      const bool joint = kPaged && both;
      const int t0 = kPaged ? 0 : t, width = joint ? D / 2 : D, d0 = joint ? t * width : 0;
      float f0 = 1.f, f1 = 0.f, all = sum;
      const float ref = fmaf(top, c2, -kLift<T>);
      float base2 = ref;
      if (joint) {
        ex.ref[par][t][row] = ref;
        ex.sum[par][t][row] = sum;
        meet(3, 256);
        // A tile whose sum is 0 saw no key (factor -1: left out).  Every other one counts, whatever it holds: scores that
        // are not numbers leave the reference at -infinity, and an infinite value may have a weight that underflows.
        const float m0 = ex.ref[par][0][row], m1 = ex.ref[par][1][row];
        const float sum0 = ex.sum[par][0][row], sum1 = ex.sum[par][1][row];
        base2 = fmaxf(m0, m1);
        f0 = sum0 == 0.f ? -1.f : exp2_approx(m0 - base2);
        f1 = sum1 == 0.f ? -1.f : exp2_approx(m1 - base2);
        all = weighed(sum0, f0) + weighed(sum1, f1);
      }
      wait(&sh.o_full[0], used[0] & 1);  // (by both tiles, item by item, so that neither falls a phase behind)
      if (joint || t0 == 1) wait(&sh.o_full[1], used[1] & 1);
      sv::tc_fence_after_sync();
      if (alive) {
        const bool none = all == 0.f;
        const float inv = whole && !none ? 1.f / all : 1.f;
        const int prow = kPaged ? 0 : t * kBlock;
        const uint32_t from = tmem + Sh::kO + t0 * D + lanes;
        const int row0 = row & ~31;  // the warp's first row
        // A thread holds a row; the warp passes 64 bytes of each of its rows through shared memory, so that a store
        // covers whole sectors of eight rows instead of pieces of 32.
        uint4* stage = ex.rows[warp];
        const int sub = lane >> 2, piece = lane & 3;  // in a store: row 8 k + sub, 16 bytes
        int at_row[4];                                // rows of out (whole) or of the partial rows, from the base
        const long long base_row = whole ? (static_cast<long long>(s.q0) + tok0) * a.heads + at.kvh * a.G : slot + prow;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = row0 + 8 * k + sub;
          at_row[k] = r >= rows ? -1 : (whole ? r / a.G * a.heads + r % a.G : r);
        }
        auto put = [&](uint4 v, int c) { stage[lane * 4 + (c ^ (lane >> 1 & 3))] = v; };
        auto flush = [&](char* base, int pitch) {  // base: the 64 bytes' place in base_row
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = 8 * k + sub;
            const uint4 v = stage[r * 4 + (piece ^ (r >> 1 & 3))];
            if (at_row[k] >= 0)
              *reinterpret_cast<uint4*>(base + static_cast<long long>(at_row[k]) * pitch + piece * 16) = v;
          }
          __syncwarp();
        };
        if (kPaged && rows <= 16) {  // few rows: each thread its own
          const long long mine = base_row + (whole ? row / a.G * a.heads + row % a.G : row);
#pragma unroll 1
          for (int d = d0; d < d0 + width; d += 32) {
            float o[32];
            sv::tmem_load_32(from + d, o);
            if (joint) {
              float o2[32];
              sv::tmem_load_32(from + D + d, o2);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = weighed(o[e], f0) + weighed(o2[e], f1);
            }
            if (row >= rows) continue;
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + mine * D + d);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  w[k] = none ? 0u : pack2(o[8 * c + 2 * k] * inv, o[8 * c + 2 * k + 1] * inv, T());
                dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
              float4* dst = reinterpret_cast<float4*>(a.part_o + mine * D + d);
#pragma unroll
              for (int c = 0; c < 8; ++c) dst[c] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
            }
          }
        } else if (whole) {
          char* base = reinterpret_cast<char*>(static_cast<T*>(a.out) + base_row * D);
#pragma unroll 1
          for (int d = d0; d < d0 + width; d += 32) {
            float o[32];
            sv::tmem_load_32(from + d, o);
            if (joint) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float o2[16];
                sv::tmem_load_16(from + D + d + 16 * h, o2);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  o[16 * h + e] = weighed(o[16 * h + e], f0) + weighed(o2[e], f1);
              }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = none ? 0u : pack2(o[8 * c + 2 * k] * inv, o[8 * c + 2 * k + 1] * inv, T());
              put(make_uint4(w[0], w[1], w[2], w[3]), c);
            }
            flush(base + d * 2, D * 2);
          }
        } else {
          char* base = reinterpret_cast<char*>(a.part_o + base_row * D);
#pragma unroll 1
          for (int d = d0; d < d0 + width; d += 16) {
            float o[16];
            sv::tmem_load_16(from + d, o);
            if (joint) {
              float o2[16];
              sv::tmem_load_16(from + D + d, o2);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = weighed(o[e], f0) + weighed(o2[e], f1);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
              put(make_uint4(__float_as_uint(o[4 * c]), __float_as_uint(o[4 * c + 1]), __float_as_uint(o[4 * c + 2]),
                             __float_as_uint(o[4 * c + 3])), c);
            flush(base + d * 4, D * 4);
          }
        }
        if (row < rows && d0 == 0) {
          if (!whole) a.part_ml[base_row + row] = make_float2(base2, all);
          else if (a.lse) a.lse[base_row + row / a.G * a.heads + row % a.G] =
              none ? -INFINITY : (base2 + log2f(all)) * kLn2;
        }
      }
      sv::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (kPaged) {
          sv::mbar_arrive(&sh.o_free[0]);
          sv::mbar_arrive(both ? &sh.o_free[1] : &sh.o_free[0]);
        } else {
          sv::mbar_arrive(&sh.o_free[t]);
        }
      }
      ++used[0];
      if (both) ++used[1];
    }
  }

  __syncwarp();
  sv::tc_fence_before_sync();
  __syncthreads();
  sv::tc_fence_after_sync();
  if (warp == kMmaWarp) sv::tmem_dealloc(tmem, Sh::kTmemCols);
  if (tid == 0 && sh.abort) report(a, -1, SPEC_ATTN_DEVERR_TIMEOUT);
}

// Joins the partial rows of every item that was cut, zeroes the rows of
// sequences found bad, and publishes the error word.  CTA (c, y) takes every
// join_split-th group of rows of the item whose first cut CTA c begins with; a
// warp takes a row: lane p weighs piece p while the pieces' columns are on their
// way.  At most one item per CTA of the main kernel is cut: a few MB of L2
// traffic, bound by two dependent loads (the record, then all the rest).
template <typename T, int D, bool kPaged>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnArgs a) {
  constexpr int kNT = kTiles<kPaged>, kE = D / 32, kWarps = kJoinThreads / 32, kFew = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sv::griddep_wait();
  sv::griddep_launch_dependents();
  const Cut cut = a.cuts[blockIdx.x];
  const int errors = a.ctrl[sv::kKvCollect];  // (the main kernel has set them all)
  const int rows = cut.active ? cut.tokens * a.G : 0;
  const int last = cut.active ? cut.shares.owner(cut.end) : 0;  // the CTA with the last piece
  for (int i = blockIdx.y * kWarps + warp; i < rows; i += a.join_split * kWarps) {
    if (kPaged && errors && a.bad[cut.b]) break;
    const int tok = i / a.G, g = i % a.G, sub = tok / a.tile_tokens;
    const int r = sub * kBlock + (tok - sub * a.tile_tokens) * a.G + g;
    // the first piece is its CTA's last segment, the others are their CTAs' first
    auto place = [&](int p) {
      return (static_cast<long long>(p) * 2 + (p == cut.first ? 1 : 0)) * (kNT * kBlock) + r;
    };
    float o[kE], ref = -INFINITY, sum = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = 0.f;
    if (last - cut.first < kFew) {  // a few pieces (most items): all at once
      float2 ml[kFew];
      float x[kFew][kE];
#pragma unroll
      for (int q = 0; q < kFew; ++q) {
        ml[q] = make_float2(-INFINITY, 0.f);
        if (cut.first + q > last) continue;
        const long long at = place(cut.first + q);
        ml[q] = a.part_ml[at];
#pragma unroll
        for (int e = 0; e < kE; e += 2) {
          const float2 v = *reinterpret_cast<const float2*>(a.part_o + at * D + lane * kE + e);
          x[q][e] = v.x;
          x[q][e + 1] = v.y;
        }
      }
#pragma unroll
      for (int q = 0; q < kFew; ++q) ref = fmaxf(ref, ml[q].x);
#pragma unroll
      for (int q = 0; q < kFew; ++q) {
        if (ml[q].y == 0.f) continue;  // no such piece, or it saw no key (a sum that is not a number counts)
        const float f = exp2_approx(ml[q].x - ref);
        sum += ml[q].y * f;
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] += x[q][e] * f;
      }
    } else {
      for (int p0 = cut.first; p0 <= last; p0 += 32) {  // (one round for up to 32 pieces)
        const float2 ml = p0 + lane <= last ? a.part_ml[place(p0 + lane)] : make_float2(-INFINITY, 0.f);
        constexpr int kAhead = 8;
        float x[kAhead][kE];
        auto fetch = [&](int q0) {
#pragma unroll
          for (int q = 0; q < kAhead; ++q) {
            if (q0 + q > last) continue;
            const float* from = a.part_o + place(q0 + q) * D + lane * kE;
#pragma unroll
            for (int e = 0; e < kE; e += 2) {
              const float2 v = *reinterpret_cast<const float2*>(from + e);
              x[q][e] = v.x;
              x[q][e + 1] = v.y;
            }
          }
        };
        fetch(p0);
        float top = ml.x;
#pragma unroll
        for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        top = fmaxf(top, ref);
        const float f = ml.y == 0.f ? -1.f : exp2_approx(ml.x - top);
        const float keep = sum == 0.f ? -1.f : exp2_approx(ref - top);
        ref = top;
        sum = weighed(sum, keep);
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] = weighed(o[e], keep);
        const float l = weighed(ml.y, f);
        const int n = min(32, last - p0 + 1);
        for (int p = 0; p < n; p += kAhead) {
          if (p > 0) fetch(p0 + p);
#pragma unroll
          for (int q = 0; q < kAhead; ++q) {
            const float w = __shfl_sync(0xffffffffu, f, (p + q) & 31);
            sum += __shfl_sync(0xffffffffu, l, (p + q) & 31);  // (0 behind the last piece)
            if (!(w < 0.f)) {  // (none behind the last piece)
#pragma unroll
              for (int e = 0; e < kE; ++e) o[e] += x[q][e] * w;
            }
          }
        }
      }
    }
    const bool none = sum == 0.f;
    const float inv = none ? 0.f : 1.f / sum;
    const long long orow = cut.row + static_cast<long long>(tok) * a.heads + g;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + orow * D + lane * kE);
#pragma unroll
    for (int e = 0; e < kE; e += 2) dst[e / 2] = none ? 0u : pack2(o[e] * inv, o[e + 1] * inv, T());
    if (a.lse && lane == 0) a.lse[orow] = none ? -INFINITY : (ref + log2f(sum)) * kLn2;
  }
  if (errors == 0) {  // (the same answer in every CTA)
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.ctrl[sv::kKvErr] = 0;
    return;
  }
  if (kPaged) {
    for (int b = blockIdx.x * a.join_split + blockIdx.y; b < a.B; b += gridDim.x * a.join_split) {
      if (!a.bad[b]) continue;
      const int n = a.len_k ? a.len_k[b] : a.S;
      const long long count = static_cast<long long>(n < 0 || n > a.S ? a.S : n) * a.heads;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + static_cast<long long>(b) * a.S * a.heads * D);
      for (long long i = threadIdx.x; i < count * D / 8; i += kJoinThreads) dst[i] = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (long long i = threadIdx.x; i < count; i += kJoinThreads)
          a.lse[static_cast<long long>(b) * a.S * a.heads + i] = -INFINITY;
    }
  }
  // the last CTA leaves the marks ready for the next call
  __shared__ int s_last;
  __syncthreads();
  if (threadIdx.x == 0) s_last = sv::kv_last_cta(a.ctrl);
  __syncthreads();
  if (!s_last) return;
  if (kPaged)
    for (int b = threadIdx.x; b < a.B; b += kJoinThreads) a.bad[b] = 0;
  __syncthreads();
  if (threadIdx.x == 0) sv::kv_publish(a.ctrl);
}

// --------------------------------------------------------------------- host
bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

bool heads_ok(int heads, int kv_heads, int head_dim, int dtype) {
  return (head_dim == 64 || head_dim == 128) && kv_heads >= 1 && heads >= kv_heads && heads <= 1024 &&
         heads % kv_heads == 0 && heads / kv_heads <= 64 && (dtype == SPEC_ATTN_BF16 || dtype == SPEC_ATTN_FP16);
}

// (The kernel works with scale * log2 e, in f32.)
bool scale_ok(float scale) { return scale > 0.f && std::isfinite(scale * kLog2e); }

bool stride_ok(int64_t stride, int heads, int head_dim) {
  return stride % 8 == 0 && stride >= static_cast<int64_t>(heads) * head_dim && stride <= (1ll << 31);
}

constexpr int64_t kMaxTokens = 1 << 24;
constexpr int kMaxBatch = 65535;

bool kv_dims_ok(const spec_kv_attn_dims& d) {
  return heads_ok(d.heads, d.kv_heads, d.head_dim, d.dtype) && d.B >= 1 && d.B <= kMaxBatch && d.S >= 1 &&
         d.S <= kMaxTree && static_cast<int64_t>(d.B) * d.S <= kMaxTokens && d.page_size >= 1 && d.num_pages >= 1 &&
         d.max_pages >= 1 && static_cast<int64_t>(d.max_pages) * d.page_size < (1ll << 31) &&
         static_cast<int64_t>(d.num_pages) * d.page_size < (1ll << 31) && stride_ok(d.q_stride, d.heads, d.head_dim);
}

bool prompt_dims_ok(const spec_prompt_dims& d) {
  return heads_ok(d.heads, d.kv_heads, d.head_dim, d.dtype) && d.B >= 1 && d.B <= kMaxBatch && d.total_q >= 1 &&
         d.total_q <= kMaxTokens && d.total_k >= 1 && d.total_k <= kMaxTokens &&
         stride_ok(d.q_stride, d.heads, d.head_dim) && stride_ok(d.k_stride, d.kv_heads, d.head_dim) &&
         stride_ok(d.v_stride, d.kv_heads, d.head_dim);
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
  size_t bad, cuts, part_ml, part_o, total;
};

// The control words and the marks, which a call expects to be zero and leaves so, lie in front and take the same bytes
// for every call: a workspace may serve calls of different batches and of both operators.  What is behind them is
// written before it is read.
Layout layout(int head_dim, int tiles) {
  Layout l;
  const size_t rows = static_cast<size_t>(kMaxGrid) * 2 * tiles * kBlock;
  l.bad = sv::kKvCtrlBytes;
  l.cuts = l.bad + up(4 * static_cast<size_t>(kMaxBatch));
  l.part_ml = l.cuts + up(sizeof(Cut) * kMaxGrid);
  l.part_o = l.part_ml + up(sizeof(float2) * rows);
  l.total = l.part_o + up(sizeof(float) * rows * head_dim);
  return l;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// A 16-bit tensor with boxes of 64 elements (128 bytes, 128-byte swizzle) by box[1], .., zeros outside; strides in
// bytes, from the second dimension on.
bool encode(CUtensorMap* map, int dtype, const void* base, int rank, const cuuint64_t (&dims)[4],
            const cuuint64_t (&strides)[3], const cuuint32_t (&box)[4]) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return fn(map, dtype == SPEC_ATTN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
            const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_tokens(CUtensorMap* map, int dtype, const void* base, int head_dim, int heads, int64_t tokens,
                   int64_t stride, int box_heads, int box_tokens) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens), 1};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(head_dim) * 2, static_cast<cuuint64_t>(stride) * 2, 0};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens), 1};
  return encode(map, dtype, base, 3, dims, strides, box);
}

template <typename T, int D, bool kPaged>
spec_status launch(const AttnArgs& a, const CUtensorMap (&maps)[3], const sv::DeviceInfo& dev, cudaStream_t s) {
  using Sh = Shape<D, kPaged>;
  constexpr size_t kBytes = 1024 + Sh::kQBytes + Sh::kStages * Sh::kTileBytes + (sizeof(Sync) + 15) / 16 * 16 +
                            sizeof(Exchange) + (kPaged ? sizeof(TreeShared) : 0);
  static_assert(kBytes <= 232448, "shared memory of one CTA");
  static_assert(kBytes > 116 * 1024, "one CTA per SM: it takes all of the tensor memory");
  static bool done[64] = {false};
  if (!done[dev.device]) {
    if (cudaFuncSetAttribute(attn_kernel<T, D, kPaged>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kBytes)) != cudaSuccess)
      return SPEC_ERR_CUDA;
    done[dev.device] = true;
  }
  const int grid = dev.sm_count < kMaxGrid ? dev.sm_count : kMaxGrid;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attn_kernel<T, D, kPaged>, a, maps[0], maps[1], maps[2]) != cudaSuccess)
    return SPEC_ERR_CUDA;
  if (sv::launch_dependent(attn_join_kernel<T, D, kPaged>, dim3(grid, a.join_split), dim3(kJoinThreads), s, a) !=
      cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

template <bool kPaged>
spec_status launch(AttnArgs& a, const CUtensorMap (&maps)[3], int head_dim, int dtype, const sv::DeviceInfo& dev,
                   void* workspace, cudaStream_t s) {
  const Layout l = layout(head_dim, kTiles<kPaged>);
  char* ws = static_cast<char*>(workspace);
  a.ctrl = reinterpret_cast<int*>(ws);
  a.bad = reinterpret_cast<int*>(ws + l.bad);
  a.cuts = reinterpret_cast<Cut*>(ws + l.cuts);
  a.part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
  a.part_o = reinterpret_cast<float*>(ws + l.part_o);
  if (dtype == SPEC_ATTN_BF16)
    return head_dim == 64 ? launch<__nv_bfloat16, 64, kPaged>(a, maps, dev, s)
                          : launch<__nv_bfloat16, 128, kPaged>(a, maps, dev, s);
  return head_dim == 64 ? launch<__half, 64, kPaged>(a, maps, dev, s) : launch<__half, 128, kPaged>(a, maps, dev, s);
}

}  // namespace

extern "C" {

size_t spec_kv_attention_workspace_bytes(spec_kv_attn_dims dims) {
  return kv_dims_ok(dims) ? layout(dims.head_dim, kTiles<true>).total : 0;
}

size_t spec_prompt_attention_workspace_bytes(spec_prompt_dims dims) {
  return prompt_dims_ok(dims) ? layout(dims.head_dim, kTiles<false>).total : 0;
}

spec_status spec_kv_attention(const void* q, const void* pool, const int32_t* block_table, const int32_t* seq_len,
                              const void* staged, const int32_t* parents, const int32_t* q_len, float scale, void* out,
                              float* out_lse, spec_kv_attn_dims dims, void* workspace, size_t workspace_bytes,
                              spec_stream_t stream) {
  if (!q || !pool || !block_table || !seq_len || !out || !workspace) return SPEC_ERR_ARG;
  if (!scale_ok(scale)) return SPEC_ERR_ARG;
  if (!kv_dims_ok(dims)) return SPEC_ERR_DIMS;
  if (misaligned(q, 16) || misaligned(pool, 16) || misaligned(staged, 16) || misaligned(out, 16) ||
      misaligned(workspace, 16) || misaligned(block_table, 4) || misaligned(seq_len, 4) || misaligned(parents, 4) ||
      misaligned(q_len, 4) || misaligned(out_lse, 4))
    return SPEC_ERR_ALIGN;
  if (workspace_bytes < spec_kv_attention_workspace_bytes(dims)) return SPEC_ERR_WORKSPACE;
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
  a.scale_log2 = scale * kLog2e;
  a.B = dims.B;
  a.S = dims.S;
  a.heads = dims.heads;
  a.kv_heads = dims.kv_heads;
  a.G = dims.heads / dims.kv_heads;
  a.page_size = dims.page_size;
  a.num_pages = dims.num_pages;
  a.max_pages = dims.max_pages;
  a.tile_tokens = kBlock / a.G;
  const int64_t tokens = static_cast<int64_t>(dims.B) * dims.S;
  CUtensorMap maps[3];
  if (!encode_tokens(&maps[0], dims.dtype, q, dims.head_dim, dims.heads, tokens, dims.q_stride, a.G, a.tile_tokens))
    return SPEC_ERR_CUDA;
  // Up to 16 rows (one token) a piece is next to nothing to join: with 1, 2 and 3 units one cache of 1000 positions took
  // 12.2, 13.6 and 14.7 us; a tree of 120 rows over 4 caches 19.0, 20.2 and 24.0 with 3, 4 and 6.
  a.least = dims.S * a.G <= 16 ? 1 : 3;
  a.join_split = dims.S * a.G <= 8 ? 1 : (dims.S * a.G < 64 ? (dims.S * a.G + 7) / 8 : 8);
  // the largest boxes that pages and blocks divide into; below eight rows (the swizzle's unit) row by row
  a.box = kBlock;
  while (a.box >= 8 && dims.page_size % a.box != 0) a.box /= 2;
  if (a.box < 8) a.box = 0;
  maps[1] = maps[0];
  if (a.box) {  // (64 columns, eight rows, the columns' places in the entry, groups of eight rows)
    const cuuint64_t entry = 2ull * dims.kv_heads * dims.head_dim;
    const cuuint64_t dim[4] = {64, 8, entry / 64, static_cast<cuuint64_t>(dims.num_pages) * dims.page_size / 8};
    const cuuint64_t stride[3] = {entry * 2, 128, entry * 16};
    const cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(dims.head_dim / 64), static_cast<cuuint32_t>(a.box / 8)};
    if (!encode(&maps[1], dims.dtype, pool, 4, dim, stride, box)) return SPEC_ERR_CUDA;
  }
  maps[2] = maps[1];  // (not used)
  return launch<true>(a, maps, dims.head_dim, dims.dtype, dev, workspace, reinterpret_cast<cudaStream_t>(stream));
}

spec_status spec_prompt_attention(const void* q, const void* k, const void* v, const int32_t* cu_q,
                                  const int32_t* cu_k, float scale, void* out, float* out_lse, spec_prompt_dims dims,
                                  void* workspace, size_t workspace_bytes, spec_stream_t stream) {
  if (!q || !k || !v || !cu_q || !out || !workspace) return SPEC_ERR_ARG;
  if (!scale_ok(scale)) return SPEC_ERR_ARG;
  if (!prompt_dims_ok(dims)) return SPEC_ERR_DIMS;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(out, 16) || misaligned(workspace, 16) ||
      misaligned(cu_q, 4) || misaligned(cu_k, 4) || misaligned(out_lse, 4))
    return SPEC_ERR_ALIGN;
  if (workspace_bytes < spec_prompt_attention_workspace_bytes(dims)) return SPEC_ERR_WORKSPACE;
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
  a.scale_log2 = scale * kLog2e;
  a.B = dims.B;
  a.heads = dims.heads;
  a.kv_heads = dims.kv_heads;
  a.G = dims.heads / dims.kv_heads;
  a.total_q = dims.total_q;
  a.total_k = dims.total_k;
  a.k_stride = dims.k_stride;
  a.v_stride = dims.v_stride;
  a.tile_tokens = kBlock / a.G;
  a.least = 6;  // (four heads over three short prompts: 18.4 us; 20.1 with 4, 23.2 with 8)
  a.join_split = 8;
  CUtensorMap maps[3];
  if (!encode_tokens(&maps[0], dims.dtype, q, dims.head_dim, dims.heads, dims.total_q, dims.q_stride, a.G,
                     a.tile_tokens) ||
      !encode_tokens(&maps[1], dims.dtype, k, dims.head_dim, dims.kv_heads, dims.total_k, dims.k_stride, 1, kBlock) ||
      !encode_tokens(&maps[2], dims.dtype, v, dims.head_dim, dims.kv_heads, dims.total_k, dims.v_stride, 1, kBlock))
    return SPEC_ERR_CUDA;
  return launch<false>(a, maps, dims.head_dim, dims.dtype, dev, workspace, reinterpret_cast<cudaStream_t>(stream));
}

spec_status spec_attention_read_error(void* workspace, int32_t* error_word, spec_stream_t stream) {
  if (!workspace || !error_word) return SPEC_ERR_ARG;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess ||
      cudaMemcpy(error_word, workspace, sizeof(int32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

}  // extern "C"
