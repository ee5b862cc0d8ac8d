// Attention over the 8-bit paged cache.  Declared in include/spec_kv8.h.
//
// A work item is a tile of up to RT query rows (row r: token r / G, head r % G of
// the group, G = heads / kv_heads) of one key-value head of one sequence.  It
// walks the keys in blocks of 128, keys in the rows of the tensor core's tiles
// and query rows in their columns, so that few rows cost little:
//   S^T = K Q^T        tcgen05.mma kind::f8f6f4, M = 128 keys, N = 3 RT (to 16)
//   P^T = exp2(S c - m) times the value's scale, one key per softmax thread
//   O^T += V^T P^T     kind::f8f6f4, M = head_dim, both read key by key (MN-major)
// The cached codes go from HBM to shared memory by TMA and from there into the
// tensor core as they are; nothing is converted.  What has more than 8 bits is
// split instead: a query row, scaled by a power of two, into three e4m3 parts
//   q = 2^t (q0 + q1 / 32 + q2 / 1024),  q0 = e4m3(q 2^-t), q1 = e4m3(32 (q 2^-t - q0)), ..
// and a weight into four, each part a group of RT columns of S, P and O; the
// products' f32 sums are put together in registers.  Three parts hold 12 bits
// of an element, down to 2^-27 of the row's largest: bf16 and fp16 queries are
// split exactly but for elements below 2^-16 of it.  Weights are rounded to fp16
// before (11 bits, as three parts would hold them; packed arithmetic takes half
// the instructions of 32-bit differences), whose subnormal end the fourth part
// reaches: weights times scale are off by 2^-25 at most where 2^-11 of them is
// less.  With three parts that was 2^-20, so that thousands of small weights were
// lost beside a large one (64 caches took 115.3 us with three, 117.1 with four).
// (Rows of the tiles that no part uses hold anything; they make columns that
// nobody reads.)
//
// Scales differ from page to page, so from key to key: a softmax thread
// multiplies its key's scores by the key's scale, and its weights by the
// value's before they are split.  Weights are w = 2^(s c - m) with a reference m
// set so that the row's largest w vs (vs the value's scale) is 2 to 4; they may
// grow to 256 (e4m3 holds 448; the parts then take steps of 32).  While all stay
// below, m does not move: the warps agree by one barrier that takes the or of
// "some weight is too large".  Otherwise the row's maxima are exchanged, m is set
// anew, and the sums and O rescaled (0.6 us).  The block after one whose largest
// weight was far above all before it (or the first) is looked through for rows
// whose weights have all become small, and m set lower for them: a row's largest
// weight may be that of a new entry, or of a cached key whose value is nearly
// zero, and what counts are the others.  (Done for every block, by an or of the
// rows' bits, it took 118 us for the 64 caches, 42 for the chains.)  Sums of the
// unsplit weights in f32 make the denominator, so what m is cancels.  m is kept
// in two parts, the rounded product of the largest score with c and the rest, so
// that scores of any size lose nothing beside it.
//
// The new tokens' entries are 16-bit and come first: their blocks take 16-bit
// products (kind::f16) of the unsplit queries and of weights rounded to the type
// of q (both operands of such a product have one type, and no more than the
// result keeps), into the first group of columns.
//
// One CTA per SM walks an equal share of all items' blocks (plus a constant per
// item).  An item cut between CTAs leaves normalised partial rows with their
// references and sums, which a second, small kernel weighs and adds in the
// order of the pieces.  Lengths are read on the device only.
//
// Bound, where there are many long caches, by HBM: 64 caches of 512 to 8191
// positions (8 key-value heads of 128, 583 MB) take 115 to 124 us, 4.7 to 5.1 TB/s
// or 69 to 75 % of the measured copy; the loads alone take about 100.  The rest is
// the start and end of each CTA's items (5 to 6 us each: queries split, the first
// reference, the 16-bit block, the way out) and the join, 2.5 us.  Short calls are
// latency: one cache of 1000 positions 15 us, of 120001 54 to 58 (4.2 to 4.5 TB/s),
// chains of 5 over 8 caches 31 to 37 (the more unequal the scores of a head, the
// more often references are set), trees of 40 over 4 caches 27 to 30.  Tiles of
// many rows are bound by the instructions of a weight (a block of 128 keys takes
// 0.75 us with 8 rows, 1.2 with 32, 1.55 with 48), wide trees over short caches by
// an item's start and end (about 13 us with 48 rows).  What the choices measured
// when they were made (us):
//   a box that brings keys and values by turns, not one for each   64 caches 153, 173
//   128-byte L2 promotion, not 256 (which reads twice from HBM)    120001 positions 58, 66
//   a warpgroup for eight rows (four of the smallest tile)         chains 44, 84
//   two teams of warpgroups, taking blocks by turns, for tiles of
//     up to 16 rows, and weights in packed fp16                    chains 37, 43
//   a tile of 40 rows (80 registers a thread, not 72)              trees 26, 32
//   weights' parts column by column, eight bytes to a store        33 caches of 36363, 35 rows: 105, 114
//   P V of a block issued before the next block's scores           64 caches 155, 177
//
// What is not a number: cached codes go into the products as they are, which
// is right for what every row sees; keys behind the end are replaced by weights
// of 0 and their V rows zeroed in shared memory.  Staged values that are not
// finite are zeroed and added, at the end, to the rows that see them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "f8_codes.cuh"
#include "internal.h"
#include "kv_copy.cuh"
#include "shares.cuh"
#include "sm103_ptx.cuh"
#include "spec_kv8.h"

namespace {

using sv::quot;
using sv::Shares;
using sv::shares_of;
using sv::warp_scan;

constexpr int kBlock = 128;          // keys per block
constexpr int kLoadWarps = 3;        // each brings every third load
constexpr int kMaxGrid = 160;        // CTAs (one per SM); sizes the workspace
// An item's start and end, in blocks (sets the shares): what a CTA's time grows by with each further item of its share,
// over what it grows by with each block.  With 2 for every tile 64 caches took 136 us beside 116, trees of 40 36 beside 32.
template <int RT>
constexpr int kItemUnits = RT == 8 ? 9 : RT == 16 ? 6 : 4;
constexpr int kMaxRows = 48;         // rows of the largest tile
constexpr int kMaxTree = 256;
constexpr int kMaxBatch = 65535;
constexpr int kMaxSlots = 8;
constexpr int kMaxGroups = kMaxRows / 8;  // softmax warpgroups (of either kind of tile)
constexpr int kMaxThreads = 32 * (4 * kMaxGroups + 1 + kLoadWarps);
constexpr int kJoinThreads = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLargest = 3.4028235e38f;
// The largest weight times scale in P where a reference is set, and ever.  (Set to 16 weights would be good to 2^-28 of the
// row's largest instead of 2^-26, but 33 chains of 5 with 7 heads would take 117 us for 111, as it is exceeded more often.)
constexpr float kSet = 4.f, kMost = 256.f;
// Where values are (nearly) zero the weights alone set the reference: at most 2^88 there and 2^96 ever, of which 2^31 can
// be added.  Where they are large weights get down to 2^-96.
constexpr float kWeightShare = 3.2311743e-27f;  // 2^-88: kMost times its inverse is 2^96
constexpr float kLogUp = 88.f, kLogDown = 96.f;
// New entries come first, and their values' scale is 1; a cached one's is the largest magnitude over 448 or 57344.  Their
// weights are 16-bit operands, which hold larger ones: references are set so that the first cached block of values of about
// unit size has its weights near the middle of what P takes.
constexpr float kSetNew4 = 64.f, kSetNew5 = 8192.f, kMostNew = 32768.f;  // (e4m3, e5m2; fp16 holds 65504)
// Where references have risen by 2^kRise since that was last done (or have been set at first), the next cached block is
// looked through: a row none of whose weights times scale is as large as kLeast has its reference set anew as well, so that
// they are off by 2^-17 of the block's largest at most.  What is in O grows by that, by 2^kGrowth at most altogether (what is
// smaller still counts for nothing in f32).
constexpr float kLeast = 0.00390625f, kGrowth = 32.f, kRise = 10.f;

// What a join needs to know of an item that was cut, left by the CTA with its first piece.
struct Cut {
  int active;
  int last;            // the CTA with its last piece
  int b, rows, row0;   // the sequence, the item's rows, the first one's index in the sequence's group
  long long base;      // the row of out of token 0's first head of the group
};

struct Args {
  const void* q;
  const void* staged;
  const uint8_t* pool;
  const float* scales;
  const int32_t* bt;
  const int32_t* len;
  const int32_t* q_len;
  const int32_t* parents;
  void* out;
  float* lse;
  float scale_log2;
  int B, S, heads, kv_heads, G, page_size, num_pages, max_pages, format, bf16;
  uint32_t page_mul, page_shift;  // p / page_size = p * page_mul >> page_shift
  int fresh_box;       // rows of one box of staged entries (a multiple of 8)
  int box;             // rows of one page box (a divisor of the page and of a block), or 0: row by row
  int least;           // units of the smallest share
  int tile_rows;       // rows of a tile (RT, or fewer where that shares them evenly)
  int join_split;      // CTAs that share the rows of one join
  long long q_stride;
  // workspace
  int* ctrl;
  int* bad;            // [kMaxBatch] error bits of each sequence
  Cut* cuts;           // [kMaxGrid]
  float4* part_ml;     // [kMaxGrid][2][kMaxRows] (reference in log2: high and low part, sum, -)
  float* part_o;       // [kMaxGrid][2][kMaxRows][D]
};

__device__ __forceinline__ void report(const Args& a, int b, int bits) {
  if (b >= 0) atomicOr(a.bad + b, bits);
  atomicOr(a.ctrl + sv::kKvCollect, bits);
}

// One sequence: Lq new tokens behind L cached ones; nt blocks of new entries, nb blocks in all.
struct Seq {
  int Lq, L, rows, tiles, nt, nb;
};

template <int RT>
__device__ __noinline__ Seq get_seq(const Args& a, int b, int& err) {
  Seq s;
  const int L = a.len[b], n = a.q_len ? a.q_len[b] : a.S;
  err = 0;
  if (n < 0 || n > a.S || (L < 0 && n > 0)) err = SPEC_ATTN_DEVERR_LENGTH;
  else if (n > 0 && L > static_cast<long long>(a.max_pages) * a.page_size) err = SPEC_ATTN_DEVERR_CAPACITY;
  s.Lq = err ? 0 : n;
  s.L = L;
  s.rows = s.Lq * a.G;
  s.tiles = (s.rows + a.tile_rows - 1) / a.tile_rows;
  s.nt = (s.Lq + kBlock - 1) / kBlock;
  s.nb = s.nt + (L <= 0 ? 0 : (L - 1) / kBlock + 1);
  return s;
}

template <int RT>
__device__ __forceinline__ long long units_of(const Args& a, const Seq& s) {
  return static_cast<long long>(s.tiles) * a.kv_heads * (s.nb + kItemUnits<RT>);
}

// A place in the list of items.
template <int RT>
struct Cursor {
  int b, kvh, tile;
  long long start;  // first unit of the item
  Seq s;

  __device__ __noinline__ void next(const Args& a) {
    start += s.nb + kItemUnits<RT>;
    if (++tile < s.tiles) return;
    tile = 0;
    if (++kvh < a.kv_heads) return;
    kvh = 0;
    do {
      if (++b >= a.B) return;  // behind the last item; start has reached the total
      int err;
      s = get_seq<RT>(a, b, err);
    } while (s.tiles == 0);
  }
};

template <int D, int RT>
struct Shape {
  // A softmax warpgroup has RH of the tile's rows, a thread its key's scores of them.  A block's way through them is a
  // chain of waits, so small tiles have two teams that take the blocks by turns, each with a reference, sum and O of its
  // own, merged at the end of the segment.
  static constexpr int kRH = RT == 8 ? 4 : 8;
  static constexpr int kGroups = RT / kRH;             // warpgroups of a team
  static constexpr int kTeams = RT <= 16 ? 2 : 1;
  static constexpr int kSoftmaxWarps = 4 * kGroups * kTeams;
  static constexpr int kMmaWarp = kSoftmaxWarps, kLoadWarp = kMmaWarp + 1, kWarps = kLoadWarp + kLoadWarps;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kN = (3 * RT + 15) / 16 * 16;    // columns of 8-bit products
  static constexpr int kN16 = (RT + 15) / 16 * 16;      // of 16-bit ones
  static constexpr int kNP = 4 * RT;                    // of the weights' parts
  static constexpr uint32_t kTmemUsed = 2 * kN + kTeams * kNP;
  static constexpr uint32_t kTmemCols = kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  // A slot of the ring: the codes of a block, groups of eight rows of keys and of values by turns (as one box brings both),
  // or the keys or the values of a block of 16-bit entries.
  static constexpr int kSlotBytes = 2 * kBlock * D;
  static constexpr int kSlots = D == 64 ? 8 : RT == 8 ? 6 : RT <= 32 ? 5 : 4;
  static constexpr int kPBytes = kNP * kBlock > kN16 * kBlock * 2 ? kNP * kBlock : kN16 * kBlock * 2;
  static constexpr int kQBytes = kN * D, kQ16Bytes = kN16 * D * 2;
  static constexpr uint32_t kMode = D == 128 ? 2 : 4;  // rows of codes: 128 or 64 bytes, swizzled as long
  static constexpr uint32_t kGroup = 16 * D;           // bytes from eight rows of keys to the next eight
  static constexpr uint32_t kValues = 8 * D;           // from a row of keys to its values
  // byte of a row of dense codes (queries), of the keys of a slot
  static __device__ __forceinline__ int mix(int row, int byte) {
    return (((byte >> 4) ^ (D == 128 ? row & 7 : row >> 1 & 3)) << 4) + (byte & 15);
  }
  static __device__ __forceinline__ int spot(int row, int byte) { return row * D + mix(row, byte); }
  static __device__ __forceinline__ int slot_spot(int row, int byte) {
    return (row >> 3) * kGroup + (row & 7) * D + mix(row, byte);
  }
};

struct Sync {
  uint64_t full[kMaxSlots], empty[kMaxSlots], q_full, s_full[2], p_full[2], p_free[2], done;
  uint32_t tmem;
  int abort;
  Shares shares;
  int at_b, at_kvh, at_tile;
  long long at_start;
  Seq at_seq;
  long long scan[kMaxThreads / 32];
};

// Of each row of the item, for each team: what turns a score into a weight.
template <int RT, int kTeams, int kSlots>
struct Rows {
  float4 st[kTeams * RT];           // scale of the score (log2), reference (high, low part), what O has grown by (log2)
  float top[kTeams * RT];           // the reference as an unscaled score
  float ex[2][4][kTeams * RT];      // maxima of scores and of weights by [warp of the group][row]
  unsigned has[kMaxGroups][4];      // by [warpgroup][warp]
  float2 turn[kTeams * RT];         // what the row's sum and its O are multiplied by; whether there was a reference, then
                                    // whether it has risen by kRise
  float risen[kTeams * RT];         // what the reference has risen by since that was looked at (log2)
  float sum[4][kTeams * RT];
  float done[kTeams * RT];          // at the end: what O is multiplied by
  float unit[RT];                   // what a 16-bit score is multiplied by to be of the same scale
  int tok[RT];                      // the row's token
  int out[RT];                      // its row of out, from the sequence's group's first
  unsigned anc[RT][8];              // ancestors of the rows' tokens (by token of the item)
  unsigned spoiled[kMaxTree / 32];  // staged entries with values that are not finite
  float scale[kSlots][2][kBlock];  // [slot] of its keys and of their values
};

// A wait that gives up after kWaitLimitNs, or as soon as another warp has.
// The CTA then runs on to its end without waiting (its results are void, the
// error word says so), so that no barrier is left with a warp missing.
// (Code that runs seldom is kept out of line or rolled: four roles share the instruction cache.  With all of it inline the
// kernels had 180 to 300 KB, and a block of the smallest tile took 2000 clocks instead of 1200.)
__device__ __noinline__ void await_long(Sync& sh, uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = sv::global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (sv::mbar_try_wait(bar, parity)) return;
    if (*reinterpret_cast<volatile int*>(&sh.abort)) return;
    if (sv::global_timer_ns() - t0 > sv::kWaitLimitNs) *reinterpret_cast<volatile int*>(&sh.abort) = 1;
  }
}
__device__ __forceinline__ void await(Sync& sh, uint64_t* bar, uint32_t parity) {
  if (!sv::mbar_try_wait(bar, parity)) await_long(sh, bar, parity);
}
__device__ __forceinline__ bool aborted(Sync& sh) { return *reinterpret_cast<volatile int*>(&sh.abort) != 0; }

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Named barriers: 1 + w the 128 threads of softmax warpgroup w, kAll those of all warpgroups.
constexpr int kAll = 15;
__device__ __forceinline__ void meet(int id, int threads) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The same, and whether any thread says so.
__device__ __forceinline__ bool meet_any(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}
// 16 bytes global -> shared, zeros where `bytes` is 0 (the address is not read then).
__device__ __forceinline__ void copy_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
// Keeps subnormal results: what a whole piece of an item counts for may be as small as the smallest outputs.
__device__ __forceinline__ float exp2_small(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The largest of three values, or not a number.
__device__ __forceinline__ float max_or_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// The largest of the warp's values; what is not a number does not count.
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// log2 of a positive x, rounded down.
__device__ __forceinline__ int ilog2(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 127; }
// Beyond 2^96 a scale would leave weights no room in f32: its rows become NaN.
__device__ __forceinline__ float value_scale(float scale, bool inside) {
  return !inside ? 0.f : scale <= 7.9228163e28f ? scale : NAN;
}
__device__ __forceinline__ void st_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void st_u16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(static_cast<unsigned short>(v)) : "memory");
}

// 16-bit values as the type of q says.
__device__ __forceinline__ float wide(uint32_t half, int bf16) {
  return bf16 ? __uint_as_float(half << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(half)));
}
__device__ __forceinline__ uint32_t narrow(float x, int bf16) {
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}
__device__ __forceinline__ bool odd_half(uint32_t half, int bf16) {
  const uint32_t inf = bf16 ? 0x7f80u : 0x7c00u;
  return (half & inf) == inf;
}

// Instruction descriptors, f32 accumulators, A = keys or values, B = queries or weights; a_mn, b_mn: A, B is MN-major.
__device__ __forceinline__ uint32_t idesc(uint32_t fmt_a, uint32_t fmt_b, uint32_t n, uint32_t a_mn, uint32_t b_mn = 0) {
  return (1u << 4) | (fmt_a << 7) | (fmt_b << 10) | (a_mn << 15) | (b_mn << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

template <int RT>
__device__ __forceinline__ void begin_at(const Args& a, Sync& sh, const Seq& s, int b, long long before, long long u) {
  const long long per_item = s.nb + kItemUnits<RT>, item = quot(u - before, per_item);
  sh.at_b = b;
  sh.at_kvh = static_cast<int>(quot(item, s.tiles));
  sh.at_tile = static_cast<int>(item - static_cast<long long>(sh.at_kvh) * s.tiles);
  sh.at_start = before + item * per_item;
  sh.at_seq = s;
}

// Where this CTA's share begins: up to 32 sequences by one warp,
template <int RT>
__device__ __noinline__ void scan_few(const Args& a, Sync& sh) {
  const int lane = threadIdx.x & 31;
  Seq s;
  s.tiles = 0;
  long long units = 0;
  if (lane < a.B) {
    int err;
    s = get_seq<RT>(a, lane, err);
    units = units_of<RT>(a, s);
    if (err && blockIdx.x == 0) report(a, lane, err);
  }
  const long long x = warp_scan(units, lane);
  const Shares shares = shares_of(__shfl_sync(0xffffffffu, x, 31), gridDim.x, a.least);
  const long long u = shares.before(blockIdx.x);
  if (lane == 0) sh.shares = shares;
  if (units > 0 && x - units <= u && u < x) begin_at<RT>(a, sh, s, lane, x - units, u);
}

// more by the whole CTA (in two passes where a thread has more than one).
template <int RT>
__device__ __noinline__ void scan_many(const Args& a, Sync& sh) {
  constexpr int kThreads = Shape<128, RT>::kThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool once = a.B <= kThreads;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    long long seen = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
      const int b = b0 + tid;
      long long units = 0;
      Seq s;
      s.tiles = 0;
      if (b < a.B) {
        int err;
        s = get_seq<RT>(a, b, err);
        units = units_of<RT>(a, s);
        if (err && pass == 0 && blockIdx.x == 0) report(a, b, err);
      }
      const long long x = warp_scan(units, lane);
      __syncthreads();
      if (lane == 31) sh.scan[warp] = x;
      __syncthreads();
      long long before = seen, sum = 0;
#pragma unroll 1
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sh.scan[w];
        sum += sh.scan[w];
      }
      seen += sum;
      if (pass == 1 || once) {
        if (once) {
          if (tid == 0) sh.shares = shares_of(seen, gridDim.x, a.least);
          __syncthreads();
        }
        const long long u = sh.shares.before(blockIdx.x), end = before + x;
        if (units > 0 && end - units <= u && u < end) begin_at<RT>(a, sh, s, b, end - units, u);
      }
    }
    if (once) return;
    if (pass == 0) {
      __syncthreads();
      if (tid == 0) sh.shares = shares_of(seen, gridDim.x, a.least);
      __syncthreads();
    }
  }
}

// The values that are not finite in column d of the spoiled entries that token `tok` sees (its ancestors, or those up to it).
template <int D>
__device__ __noinline__ float spoiled_sum(const Args& a, int b, int kvh, int n, int tok, int d, const unsigned* spoiled,
                                          const unsigned* anc) {
  float sum = 0.f;
#pragma unroll 1
  for (int m = 0; m < n; ++m) {
    if (!(spoiled[m >> 5] >> (m & 31) & 1u)) continue;
    if (!(anc ? anc[m >> 5] >> (m & 31) & 1u : m <= tok)) continue;
    const uint32_t v = static_cast<const uint16_t*>(
        a.staged)[((static_cast<long long>(b) * a.S + m) * 2 * a.kv_heads + a.kv_heads + kvh) * D + d];
    if (odd_half(v, a.bf16)) sum += wide(v, a.bf16);
  }
  return sum;
}

template <int D, int RT>
__global__ void __launch_bounds__(Shape<D, RT>::kThreads, 1)
    kv8_attn_kernel(const Args a, const __grid_constant__ CUtensorMap map_pool,
                    const __grid_constant__ CUtensorMap map_staged) {
  using Sh = Shape<D, RT>;
  constexpr int RH = Sh::kRH, kThreads = Sh::kThreads, kMmaWarp = Sh::kMmaWarp, kLoadWarp = Sh::kLoadWarp;
  constexpr int kSoftmaxWarps = Sh::kSoftmaxWarps;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem;
  uint8_t* p_tile = ring + Sh::kSlots * Sh::kSlotBytes;  // two
  uint8_t* q_tile = p_tile + 2 * Sh::kPBytes;
  uint8_t* q16_tile = q_tile + Sh::kQBytes;
  uint8_t* tail = q16_tile + Sh::kQ16Bytes;
  Sync& sh = *reinterpret_cast<Sync*>(tail);
  auto& rw = *reinterpret_cast<Rows<RT, Sh::kTeams, Sh::kSlots>*>(tail + (sizeof(Sync) + 15) / 16 * 16);
  // (the shuffle tells the compiler that the warp index is the same in all lanes)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int cta = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < Sh::kSlots; ++i) {
      sv::mbar_init(&sh.full[i], 33);  // (a warp's copies, and its bulk copies' bytes)
      sv::mbar_init(&sh.empty[i], 1);
    }
    sv::mbar_init(&sh.q_full, kSoftmaxWarps);
    for (int t = 0; t < 2; ++t) {
      sv::mbar_init(&sh.s_full[t], 1);
      sv::mbar_init(&sh.p_full[t], 4 * Sh::kGroups);
      sv::mbar_init(&sh.p_free[t], 1);
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
    if (a.box) sv::prefetch_tensor_map(&map_pool);
    sv::prefetch_tensor_map(&map_staged);
  }
  // up to here nothing of the caller's was touched: what came before on the stream may still run
  sv::griddep_wait();
  sv::griddep_launch_dependents();
  if (tid == 0) a.cuts[cta].active = 0;
  if (a.B > 32) scan_many<RT>(a, sh);
  else if (warp == 0) scan_few<RT>(a, sh);
  if (a.parents) {  // trees are checked once per sequence
    for (int b = cta; b < a.B; b += gridDim.x) {
      int err;
      const Seq s = get_seq<RT>(a, b, err);
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
  Cursor<RT> at = {};
  at.start = u1;  // no share: nothing to walk
  if (u0 < u1) {
    at.b = sh.at_b;
    at.kvh = sh.at_kvh;
    at.tile = sh.at_tile;
    at.start = sh.at_start;
    at.s = sh.at_seq;
  }

  if (warp >= kLoadWarp) {
    // ------------------------------------------------------------- loads
    uint32_t loads = 0;
    const uint64_t policy = a.S * a.G <= RT ? sv::l2_policy_evict_first() : sv::l2_policy_evict_normal();
    const int lw = warp - kLoadWarp;
    const bool issuer = elect_one();
    constexpr int kEach = kBlock / 32;
    auto room = [&](uint32_t load) -> uint32_t {  // waits until a load's slot is free
      const uint32_t slot = load % Sh::kSlots;
      await(sh, &sh.empty[slot], (load / Sh::kSlots & 1) ^ 1);
      return slot;
    };
    // The warps take the loads by turns.  A wait by parity is right only while the slot is at most one round behind.  So
    // slots are given back in the order of the loads (new entries' keys with their values, though they are done with
    // sooner), and a warp's last load, whose slot was free, lies within the ring of its next one: the slot's last round but
    // one has then been given back.
    static_assert(kLoadWarps < Sh::kSlots, "a warp's next load lies within the ring");
    uint32_t mine = lw;  // this warp's next load
    for (; at.start < u1; at.next(a)) {
      const int lo = static_cast<int>(max(0ll, u0 - at.start - kItemUnits<RT>));
      const int hi = static_cast<int>(min(static_cast<long long>(at.s.nb), u1 - at.start - kItemUnits<RT>));
      if (hi <= lo) continue;
      const int tails = max(0, min(at.s.nt, hi) - lo);
      const int* table = a.bt + static_cast<long long>(at.b) * a.max_pages;
      // The positions of block j that this lane looks up: lane, lane + 32, .. (as boxes, also its box's first); their
      // pages are fetched one load of this warp, three loads of the CTA, ahead.  kNone: zeros.
      constexpr int kNone = -0x7fffffff - 1;
      auto col_of = [&](int p) { return static_cast<int>(static_cast<uint64_t>(p) * a.page_mul >> a.page_shift); };
      auto fetch = [&](int j, int (&page)[kEach], int& first) {
        const int p0 = (j - at.s.nt) * kBlock;
        const bool cached = j >= at.s.nt && j < hi;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const int p = p0 + 32 * e + lane;
          page[e] = cached && p < at.s.L ? table[col_of(p)] : kNone;
        }
        const int p = p0 + lane * a.box;
        first = cached && a.box && lane * a.box < kBlock && p < at.s.L ? table[col_of(p)] : kNone;
      };
      int page[kEach], next[kEach], first = kNone, next_first = kNone;
      const int count = (hi - lo) + tails;
      auto block_of = [&](int n) { return lo + (n < 2 * tails ? n / 2 : n - tails); };
      int n = static_cast<int>(mine - loads);
      fetch(block_of(n), next, next_first);
      for (; n < count; n += kLoadWarps, mine += kLoadWarps) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) page[e] = next[e];
        first = next_first;
        fetch(block_of(n + kLoadWarps), next, next_first);
        const int j = block_of(n);
        const uint32_t load = loads + n;
        if (n < 2 * tails) {  // 16-bit entries: a slot of keys, a slot of values
          const uint32_t slot = room(load);
          if (__any_sync(0xffffffffu, aborted(sh))) continue;
          if (issuer) {
            sv::mbar_arrive_expect_tx(&sh.full[slot], a.fresh_box * D * 2);
            const int tok = at.b * a.S + j * kBlock, head = (n & 1) * a.kv_heads + at.kvh;
            uint8_t* dst = ring + slot * Sh::kSlotBytes;
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              sv::tma_load_3d(dst + h * 16384, &map_staged, &sh.full[slot], h * 64, head, tok, policy);
          }
          __syncwarp();
          sv::mbar_arrive(&sh.full[slot]);
          continue;
        }
        const int p0 = (j - at.s.nt) * kBlock, valid = min(kBlock, at.s.L - p0);
        int row[kEach];  // where a position's page does not exist: zeros, and the sequence is refused
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          row[e] = -1;
          if (page[e] == kNone) continue;
          const int p = p0 + 32 * e + lane;
          if (page[e] >= 0 && page[e] < a.num_pages) row[e] = page[e] * a.page_size + (p - col_of(p) * a.page_size);
          else report(a, at.b, SPEC_ATTN_DEVERR_PAGE);
        }
        const uint32_t slot = room(load);
        if (__any_sync(0xffffffffu, aborted(sh))) continue;
        uint8_t* dst = ring + slot * Sh::kSlotBytes;
        if (a.box) {
          const int boxes = (valid + a.box - 1) / a.box, p = p0 + lane * a.box;
          // groups of eight rows of the pool (behind it the box finds zeros)
          const int group = first >= 0 && first < a.num_pages
                                ? (first * a.page_size + (p - col_of(p) * a.page_size)) / 8 : a.num_pages * a.page_size / 8;
          if (issuer) sv::mbar_arrive_expect_tx(&sh.full[slot], boxes * a.box * 2 * D);
          __syncwarp();
#pragma unroll 1
          for (int i0 = 0; i0 < boxes; i0 += 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int at_group = __shfl_sync(0xffffffffu, group, i0 + i);
              if (issuer && i0 + i < boxes)
                sv::tma_load_5d(dst + (i0 + i) * a.box * 2 * D, &map_pool, &sh.full[slot], 0, 0, 0, at_group, at.kvh, policy);
            }
          }
          __syncwarp();
        } else {
          constexpr int kPieces = D / 16, kAtOnce = 32 / kPieces;  // 16-byte pieces of a row, rows per instruction
          const uint32_t to = sv::smem_u32(dst);
          const int piece = lane % kPieces, sub = lane / kPieces;
          const uint8_t* from = a.pool + static_cast<long long>(at.kvh) * D + piece * 16;
          const unsigned long long entry = 2ull * a.kv_heads * D;
#pragma unroll 1
          for (int e = 0; e < kEach; ++e) {
            const int mine_row = e == 0 ? row[0] : e == 1 ? row[1] : e == 2 ? row[2] : row[3];
#pragma unroll
            for (int i = 0; i < 32 / kAtOnce; ++i) {
              const int in = i * kAtOnce + sub, r = __shfl_sync(0xffffffffu, mine_row, in);
              const uint8_t* src = from + static_cast<unsigned>(max(r, 0)) * entry;
              const uint32_t spot = to + Sh::slot_spot(32 * e + in, piece * 16);
              copy_16(spot, src, r < 0 ? 0 : 16);
              copy_16(spot + Sh::kValues, src + static_cast<long long>(a.kv_heads) * D, r < 0 ? 0 : 16);
            }
          }
          if (issuer) sv::mbar_arrive(&sh.full[slot]);
          __syncwarp();
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e) {  // the scales of the block's keys
          const float* src = a.scales + 2ll * (row[e] < 0 ? 0 : page[e]) * a.kv_heads + at.kvh;
          copy_4(sv::smem_u32(&rw.scale[slot][0][32 * e + lane]), src, row[e] < 0 ? 0 : 4);
          copy_4(sv::smem_u32(&rw.scale[slot][1][32 * e + lane]), src + a.kv_heads, row[e] < 0 ? 0 : 4);
        }
        copies_arrive(&sh.full[slot]);
      }
      loads += count;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (aborted(sh) && lane == 0) {  // leave no copy in flight
      const uint32_t last = loads > Sh::kSlots ? loads - Sh::kSlots : 0;
      for (uint32_t i = last; i < loads; ++i) sv::mbar_wait(&sh.full[i % Sh::kSlots], i / Sh::kSlots & 1);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // --------------------------------------------------------------- MMA
    // All lanes walk the loop, so that addresses stay in uniform registers; one issues.
    const bool issuer = elect_one();
    uint32_t loads = 0, segs = 0, uses[2] = {0, 0};  // before the segment: loads, and blocks by score tile
    const uint32_t type = a.bf16 ? 1u : 0u, fmt = static_cast<uint32_t>(a.format);
    const uint32_t id_s = idesc(fmt, 0, Sh::kN, 0), id_o = idesc(fmt, 0, Sh::kNP, 1, 1);
    const uint32_t id_s16 = idesc(type, type, Sh::kN16, 0), id_o16 = idesc(type, type, Sh::kN16, 1);
    const uint32_t ring_addr = sv::smem_u32(ring), q_addr = sv::smem_u32(q_tile), q16_addr = sv::smem_u32(q16_tile);
    const uint32_t p_addr = sv::smem_u32(p_tile);
    // descriptors of the tiles' starts; a step along K adds its bytes / 16
    const uint64_t k_desc = sv::smem_desc(0, 16, Sh::kGroup, Sh::kMode), v_desc = sv::smem_desc(0, 0, Sh::kGroup, Sh::kMode);
    const uint64_t q_desc = sv::smem_desc(q_addr, 16, 8 * D, Sh::kMode), row_desc = sv::smem_desc(0, 16, 1024, 2);
    // weights in 8-bit parts: keys 16 bytes apart, 16 columns in a row of them
    const uint64_t part_desc = sv::smem_desc(0, 128, kBlock * 16, 0);
    const uint64_t v16_desc = sv::smem_desc(0, D == 128 ? 16384 : 0, 1024, 2);  // (head_dim 64: rows 64.. repeat the first)
    auto arrived = [&](uint32_t load) -> uint32_t {  // waits for a load; its address / 16
      const uint32_t slot = load % Sh::kSlots;
      await(sh, &sh.full[slot], load / Sh::kSlots & 1);
      if (!a.box) sv::fence_proxy_async_smem();  // (rows that were copied came through the generic proxy)
      return __shfl_sync(0xffffffffu, (ring_addr + slot * Sh::kSlotBytes) >> 4, 0);
    };
    for (; at.start < u1; at.next(a)) {
      const int lo = static_cast<int>(max(0ll, u0 - at.start - kItemUnits<RT>));
      const int hi = static_cast<int>(min(static_cast<long long>(at.s.nb), u1 - at.start - kItemUnits<RT>));
      const int nb = hi - lo;
      if (nb <= 0) continue;
      const int tails = max(0, min(at.s.nt - lo, nb));  // blocks of new entries in the segment
      auto load_of = [&](int i) { return loads + i + min(i, tails); };  // the slot of block i (of its keys)
      auto scores = [&](int i) {
        const uint32_t load = load_of(i), buf = i & 1;
        const uint32_t d = __shfl_sync(0xffffffffu, tmem + buf * Sh::kN, 0);
        const uint32_t k_at = arrived(load);
        sv::tc_fence_after_sync();
        if (issuer) {
          if (i < tails) {
#pragma unroll 1
            for (int k = 0; k < D / 16; ++k)
              sv::mma_bf16_ss(d, row_desc + k_at + (((k / 4) * 16384 + (k % 4) * 32) >> 4),
                              row_desc + (q16_addr >> 4) + (((k / 4) * (Sh::kN16 * 128) + (k % 4) * 32) >> 4), id_s16, k > 0);
          } else {
#pragma unroll
            for (int k = 0; k < D / 32; ++k) sv::mma_f8_ss(d, k_desc + k_at + k * 2, q_desc + k * 2, id_s, k > 0);
          }
          sv::mma_commit(&sh.s_full[buf]);
        }
        __syncwarp();
      };
      await(sh, &sh.q_full, segs & 1);
      scores(0);
      if (nb > 1) scores(1);
#pragma unroll 1
      for (int i = 0; i < nb; ++i) {
        const bool fresh = i < tails;
        const uint32_t load = load_of(i) + (fresh ? 1 : 0), buf = i & 1;
        const uint32_t v_at = fresh ? arrived(load)
                                    : __shfl_sync(0xffffffffu, (ring_addr + load % Sh::kSlots * Sh::kSlotBytes) >> 4, 0);
        await(sh, &sh.p_full[buf], (uses[buf] + (i >> 1)) & 1);
        sv::tc_fence_after_sync();
        const uint32_t d = __shfl_sync(0xffffffffu, tmem + 2 * Sh::kN + (Sh::kTeams == 2 ? buf : 0) * Sh::kNP, 0);
        const uint32_t p = __shfl_sync(0xffffffffu, (p_addr + buf * Sh::kPBytes) >> 4, 0);
        if (issuer) {
          if (fresh) {  // (steps of 16 keys, as far as there are any)
            const int steps = (min(kBlock, at.s.Lq - (lo + i) * kBlock) + 15) / 16;
#pragma unroll 1
            for (int k = 0; k < steps; ++k)
              sv::mma_bf16_ss(d, v16_desc + v_at + k * 128,
                              row_desc + p + (((k / 4) * (Sh::kN16 * 128) + (k % 4) * 32) >> 4), id_o16, 1);
          } else {
#pragma unroll
            for (int k = 0; k < kBlock / 32; ++k)
              sv::mma_f8_ss(d, v_desc + v_at + ((Sh::kValues + k * 4 * Sh::kGroup) >> 4), part_desc + p + k * 32, id_o, 1);
          }
          sv::mma_commit(&sh.p_free[buf]);
          if (fresh) sv::mma_commit(&sh.empty[(load - 1) % Sh::kSlots]);
          sv::mma_commit(&sh.empty[load % Sh::kSlots]);
        }
        __syncwarp();
        if (i + 2 < nb) scores(i + 2);
      }
      loads += nb + tails;
      uses[0] += (nb + 1) / 2;
      uses[1] += nb / 2;
      ++segs;
    }
    if (aborted(sh)) {  // the products in flight end before the tensor memory is given back
      if (issuer) sv::mma_commit(&sh.done);
      __syncwarp();
      sv::mbar_wait(&sh.done, 0);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- softmax
    constexpr int kTeams = Sh::kTeams;
    const int group = warp >> 2, team = group / Sh::kGroups, wg = group % Sh::kGroups, quad = warp & 3;
    const int key = tid & (kBlock - 1), bar = 1 + group;
    const int own0 = team * RT + wg * RH;                      // this warpgroup's first row among the teams'
    const uint32_t lanes = static_cast<uint32_t>(quad) << 21;  // this warp's 32 TMEM lanes
    const uint32_t o_addr = tmem + 2 * Sh::kN + team * Sh::kNP + wg * RH + lanes;
    const float c2 = a.scale_log2;
    uint32_t loads = 0, uses[2] = {0, 0};
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      await(sh, bar, parity);
      __syncwarp();
    };
    auto wait_done = [&](int i) {  // the product with block i's P
      wait(&sh.p_free[i & 1], (uses[i & 1] + (i >> 1)) & 1);
      sv::tc_fence_after_sync();
    };
    for (; at.start < u1; at.next(a)) {
      const int lo = static_cast<int>(max(0ll, u0 - at.start - kItemUnits<RT>));
      const int hi = static_cast<int>(min(static_cast<long long>(at.s.nb), u1 - at.start - kItemUnits<RT>));
      const int nb = hi - lo;
      if (nb <= 0) continue;
      const Seq& s = at.s;
      const int row0 = at.tile * a.tile_rows, rows = min(a.tile_rows, s.rows - row0), tok0 = row0 / a.G;
      const int mine = rows - wg * RH;  // (rows that the tile does not have hold anything, and raise nothing)
      const int tails = max(0, min(s.nt - lo, nb));
      const bool tree = a.parents != nullptr;
      // ---- the item's queries: three 8-bit parts, and as they are
      constexpr int kE = D / 32, kMine = (RT + kSoftmaxWarps - 1) / kSoftmaxWarps;  // elements of a lane, rows of a warp
      uint32_t q[kMine][kE / 2];
      int tok_of[kMine];
#pragma unroll
      for (int n = 0; n < kMine; ++n) {
        const int r = warp + n * kSoftmaxWarps, tok = (row0 + r) / a.G, g = (row0 + r) - tok * a.G;
        tok_of[n] = tok;
        q[n][0] = q[n][kE / 2 - 1] = 0;
        if (r < rows) {
          const uint16_t* from = static_cast<const uint16_t*>(a.q) +
                                 (static_cast<long long>(at.b) * a.S + tok) * a.q_stride +
                                 (at.kvh * a.G + g) * D + lane * kE;
          if (kE == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(from);
            q[n][0] = v.x;
            q[n][kE / 2 - 1] = v.y;
          } else {
            q[n][0] = *reinterpret_cast<const uint32_t*>(from);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < kMine; ++n) {
        const int r = warp + n * kSoftmaxWarps;
        if (r >= RT) continue;
        uint32_t(&w)[kE / 2] = q[n];
        float x[kE], most = 0.f;
        bool fine = true;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          x[e] = wide(e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu, a.bf16);
          fine &= fabsf(x[e]) < 1.2676506e30f;  // 2^100
          most = fmaxf(most, fabsf(x[e]));
        }
        fine = __all_sync(0xffffffffu, fine);
        most = warp_max(most);
        // most / unit in [128, 256), unit 2^-100 at least
        const uint32_t ex = max(27, static_cast<int>(__float_as_uint(most) >> 23) - 7);
        const float unit = __uint_as_float(ex << 23), inv = __uint_as_float((254u - ex) << 23);
        uint32_t part[3] = {0, 0, 0};
        if (fine) {
#pragma unroll
          for (int e = 0; e < kE; e += 2) {
            float u = x[e] * inv, v = x[e + 1] * inv;
#pragma unroll
            for (int p = 0; p < 3; ++p) {
              const uint32_t c = sv::f8_pair_e4m3(u, v);
              part[p] |= c << (8 * e);
              const float2 back = sv::f8_values_e4m3(c);
              u = (u - back.x) * 32.f;
              v = (v - back.y) * 32.f;
            }
          }
        } else {
          part[0] = 0x7f7f7f7fu;  // not a number: neither are the row's scores
#pragma unroll
          for (int i = 0; i < kE / 2; ++i) w[i] = 0x7fff7fffu;
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          uint8_t* to = q_tile + Sh::spot(p * RT + r, lane * kE);
          if (kE == 4) *reinterpret_cast<uint32_t*>(to) = part[p];
          else *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(part[p]);
        }
        const int d = lane * kE;
        uint8_t* to = q16_tile + (d >> 6) * (Sh::kN16 * 128) + r * 128 + (((d & 63) * 2 >> 4 ^ (r & 7)) << 4) + (d * 2 & 15);
        if (kE == 4) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[kE / 2 - 1]);
        else *reinterpret_cast<uint32_t*>(to) = w[0];
        if (lane < kTeams) {
          // no reference yet: every weight is too large (of a row that the tile does not have, 0)
          rw.st[lane * RT + r] = r < rows ? make_float4(unit * c2, -INFINITY, 0.f, 0.f) : make_float4(1e-30f, INFINITY, 0.f, 0.f);
          rw.top[lane * RT + r] = -INFINITY;
        }
        if (lane == 0) {
          rw.unit[r] = inv;
          rw.tok[r] = tok_of[n];
          rw.out[r] = tok_of[n] * a.heads + (row0 + r - tok_of[n] * a.G);
        }
      }
      if (tails > 0) {
        if (tree) {  // (a node's depth in dependent loads)
          const int count = (row0 + rows - 1) / a.G - tok0 + 1;
          if (tid < count) {
            unsigned* anc = rw.anc[tid];
#pragma unroll
            for (int w = 0; w < 8; ++w) anc[w] = 0;
            int p = tok0 + tid;
            while (p >= 0) {
              anc[p >> 5] |= 1u << (p & 31);
              const int up = a.parents[static_cast<long long>(at.b) * a.S + p];
              p = up < p ? up : -1;  // (a bad parent is flagged; the walk still ends)
            }
          }
        }
        if (tid < kMaxTree / 32) rw.spoiled[tid] = 0;
      }
      {  // O starts at 0
        uint32_t z[RH];
#pragma unroll
        for (int i = 0; i < RH; ++i) z[i] = 0;
#pragma unroll
        for (int p = 0; p < 4; ++p) sv::tmem_store(o_addr + p * RT, z);
        sv::tmem_wait_st();
      }
      sv::fence_proxy_async_smem();
      meet(kAll, 32 * kSoftmaxWarps);
      if (lane == 0) sv::mbar_arrive(&sh.q_full);

      float sum[RH];
      // the rows' state, in registers where there are enough
      constexpr bool kHeld = RT == 8;
      float4 held[kHeld ? RH : 1];
#pragma unroll
      for (int i = 0; i < RH; ++i) {
        sum[i] = 0.f;
        if (kHeld) held[kHeld ? i : 0] = rw.st[own0 + i];
      }
      constexpr uint32_t kSome = 0x100, kLarge = 0x200;
      bool risen = false;  // a row's reference has, by kRise
#pragma unroll 1
      for (int i = team; i < nb; i += kTeams) {
        const int j = lo + i;
        const bool fresh = i < tails;
        const uint32_t buf = i & 1;
        const int pos = (fresh ? j : j - s.nt) * kBlock + key;
        const bool inside = pos < (fresh ? s.Lq : s.L);
        const uint32_t load = loads + i + min(i, tails) + (fresh ? 1 : 0), slot = load % Sh::kSlots;  // (V's, where K and V are two)
        // V rows behind the end are zeroed; of new entries also what is not finite (added at the end)
        const int left = (fresh ? s.Lq - j * kBlock : s.L - (j - s.nt) * kBlock);
        if (left < kBlock || (fresh && s.Lq > 1)) {
          wait(&sh.full[slot], load / Sh::kSlots & 1);
          uint8_t* tile = ring + slot * Sh::kSlotBytes;
          const int mine0 = wg * kBlock + key;  // of the team's threads
          if (fresh) {
            // 16-byte pieces of the rows that the product's steps of 16 take
            constexpr int kPieces = D / 8;
            const int end = (min(left, kBlock) + 15) / 16 * 16 * kPieces;
            const uint32_t up = a.bf16 ? 0x00800080u : 0x04000400u;  // carries a magnitude that is not finite into the sign
#pragma unroll 1
            for (int n = mine0; n < end; n += Sh::kGroups * kBlock) {
              const int row = n / kPieces, piece = n % kPieces;
              uint4* at16 = reinterpret_cast<uint4*>(tile + (piece >> 3) * 16384 + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
              if (row >= left) {
                *at16 = make_uint4(0, 0, 0, 0);
                continue;
              }
              if (s.Lq == 1) continue;  // (every row sees it: the product is right)
              const uint4 v = *at16;
              const uint32_t hit = ((v.x & 0x7fff7fffu) + up) | ((v.y & 0x7fff7fffu) + up) |
                                   ((v.z & 0x7fff7fffu) + up) | ((v.w & 0x7fff7fffu) + up);
              if (hit & 0x80008000u) {
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t odd = ((w[e] & 0x7fff7fffu) + up) & 0x80008000u;
                  if (odd & 0x8000u) w[e] &= 0xffff0000u;
                  if (odd & 0x80000000u) w[e] &= 0xffffu;
                }
                *at16 = make_uint4(w[0], w[1], w[2], w[3]);
                const int m = j * kBlock + row;
                atomicOr(&rw.spoiled[m >> 5], 1u << (m & 31));
              }
            }
          } else {
            constexpr int kPieces = D / 16;
#pragma unroll 1
            for (int n = left * kPieces + mine0; n < kBlock * kPieces; n += Sh::kGroups * kBlock)
              *reinterpret_cast<uint4*>(tile + Sh::kValues + Sh::slot_spot(n / kPieces, n % kPieces * 16)) = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }

        // (The products with P of two blocks before were issued ahead of these scores', so they are done as well.)
        wait(&sh.s_full[buf], (uses[buf] + (i >> 1)) & 1);
        sv::tc_fence_after_sync();
        if (mine <= 0) {  // a warpgroup without rows of the tile
          sv::fence_proxy_async_smem();
          sv::tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) sv::mbar_arrive(&sh.p_full[buf]);
          continue;
        }
        if (!fresh) wait(&sh.full[slot], load / Sh::kSlots & 1);  // (K has come with them)
        const float ks = rw.scale[slot][0][key], vs = fresh ? 1.f : value_scale(rw.scale[slot][1][key], inside);
        const uint32_t s_addr = tmem + buf * Sh::kN + wg * RH + lanes;
        float x[RH];  // scores (-infinity: hidden)
        {
          uint32_t s0[RH], s1[RH], s2[RH];
          sv::tmem_start(s_addr, s0);
          if (!fresh) {
            sv::tmem_start(s_addr + RT, s1);
            sv::tmem_start(s_addr + 2 * RT, s2);
          }
          sv::tmem_wait_ld();
          sv::tmem_use(s0);
          if (!fresh) {
            sv::tmem_use(s1);
            sv::tmem_use(s2);
#pragma unroll
            for (int k = 0; k < RH; ++k)
              x[k] = ks * fmaf(__uint_as_float(s2[k]), 1.f / 1024, fmaf(__uint_as_float(s1[k]), 1.f / 32, __uint_as_float(s0[k])));
            if (left < kBlock && !inside) {
#pragma unroll
              for (int k = 0; k < RH; ++k) x[k] = -INFINITY;
            }
          } else {
#pragma unroll
            for (int k = 0; k < RH; ++k) {
              const int r = wg * RH + k, tok = rw.tok[r];
              const bool sees = inside && k < mine &&
                                (tree ? rw.anc[tok - tok0][pos >> 5] >> (pos & 31) & 1u : pos <= tok);
              x[k] = sees ? __uint_as_float(s0[k]) * rw.unit[r] : -INFINITY;
            }
          }
        }
        float w[RH], largest = 0.f;  // weights
#pragma unroll
        for (int k = 0; k < RH; ++k) {
          const float4 st = kHeld ? held[kHeld ? k : 0] : rw.st[own0 + k];
          w[k] = exp2_approx(fmaf(x[k], st.x, -st.y) - st.z);
        }
#pragma unroll
        for (int k = 0; k < RH; k += 2) largest = max_or_nan(largest, w[k], w[k + 1]);
        // too large times the value's scale, or alone: then beyond 2^96
        bool set = !(largest * (vs + kWeightShare) <= (fresh ? kMostNew : kMost));
        const bool check = risen && !fresh;
        if (check) {  // .. or all too small: the rows of which a warp has found a weight of kLeast, a bit each
          uint32_t has = set ? kLarge : 0u;
#pragma unroll
          for (int k = 0; k < RH; ++k) has |= k >= mine || w[k] * vs >= kLeast ? 1u << k : 0u;
          if (largest * vs != 0.f) has |= kSome;
          has = __reduce_or_sync(0xffffffffu, has);
          if (lane == 0) rw.has[group][quad] = has;
          meet(bar, 128);
          has = rw.has[group][0] | rw.has[group][1] | rw.has[group][2] | rw.has[group][3];
          set = has >= kLarge || (has & kSome && (has & (kSome - 1)) != (1u << RH) - 1);
        } else {
          set = meet_any(bar, 128, set);
        }
        if (check) risen = false;
        if (set) {
          // ---- references anew; between the barriers a thread per row does what is the row's
          const int own = own0 + key;
#pragma unroll
          for (int k = 0; k < RH; ++k) {
            const float m = warp_max(x[k]);  // (NaN in all lanes: counts as -infinity)
            if (lane == 0) rw.ex[0][quad][own0 + k] = fmaxf(m, -INFINITY);
          }
          meet(bar, 128);
          float old2 = 0.f, old3 = 0.f;
          if (key < RH) {
            const float4 st = rw.st[own];
            const float old = rw.top[own];
            const float top = fmaxf(fmaxf(fmaxf(rw.ex[0][0][own], rw.ex[0][1][own]),
                                          fmaxf(rw.ex[0][2][own], rw.ex[0][3][own])), old);
            old2 = st.y;
            old3 = st.z;
            rw.turn[own].y = old == -INFINITY;
            // A row that has seen nothing but scores of -infinity has no reference yet: they weigh nothing against the least
            // finite one, and the first other score weighs too much.
            if (key < mine) {
              rw.st[own].y = top == -INFINITY ? -kLargest : top * st.x;
              rw.st[own].z = top == -INFINITY ? 0.f : fmaf(top, st.x, -(top * st.x));
            }
            rw.top[own] = top;
          }
          meet(bar, 128);
#pragma unroll
          for (int k = 0; k < RH; ++k) {
            const float4 st = rw.st[own0 + k];
            const float m = warp_max(exp2_approx(fmaf(x[k], st.x, -st.y) - st.z) * vs);
            if (lane == 0) rw.ex[1][quad][own0 + k] = fmaxf(m, 0.f);
          }
          meet(bar, 128);
          if (key < RH) {
            const float4 st = rw.st[own];
            const bool none = rw.turn[own].y != 0.f;
            const float most = fmaxf(fmaxf(rw.ex[1][0][own], rw.ex[1][1][own]), fmaxf(rw.ex[1][2][own], rw.ex[1][3][own]));
            // the factor, a power of two, goes into the reference's low part
            const float set = !fresh ? kSet : a.format ? kSetNew5 : kSetNew4;
            float low = st.z - (most > 0.f ? static_cast<float>(ilog2(__fdividef(set, most))) : kLogUp);
            low = fminf(fmaxf(low, st.z - kLogUp), st.z + kLogDown);
            float turn = 0.f, grown = 0.f, risen = kRise;
            if (!none) {
              const float old = (old2 - st.y) + old3;  // the old reference beside the new high part
              if (low < old)  // what is in O and in the sum grows for blocks of small weights only
                low = check && !(most * exp2_approx(st.z - old) >= kLeast) ? fmaxf(low, old - (kGrowth - st.w)) : old;
              grown = fmaxf(st.w + (old - low), 0.f);
              risen = rw.risen[own] + (low - old);
              turn = exp2_approx(old - low);
            }
            if (key < mine) {
              rw.st[own].z = low;
              rw.st[own].w = grown;
            }
            rw.turn[own] = make_float2(turn, key < mine && risen >= kRise);
            rw.risen[own] = risen >= kRise ? 0.f : fmaxf(risen, 0.f);
          }
          if (i >= kTeams) wait_done(i - kTeams);  // O as it stands takes the new units
          meet(bar, 128);
#pragma unroll
          for (int k = 0; k < RH; ++k) {
            const float4 st = rw.st[own0 + k];
            const float2 turn = rw.turn[own0 + k];
            if (kHeld) held[kHeld ? k : 0] = st;
            sum[k] *= turn.x;
            risen |= turn.y != 0.f;
            w[k] = exp2_approx(fmaf(x[k], st.x, -st.y) - st.z);
          }
          if (i >= kTeams) {
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
              uint32_t o[RH];
              sv::tmem_start(o_addr + g * RT, o);
              sv::tmem_wait_ld();
              sv::tmem_use(o);
#pragma unroll
              for (int n = 0; n < RH; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * rw.turn[own0 + n].x);
              sv::tmem_store(o_addr + g * RT, o);
            }
            sv::tmem_wait_st();
          }
        }
#pragma unroll
        for (int k = 0; k < RH; ++k) sum[k] += w[k];
        // ---- P
        const uint32_t p_addr = sv::smem_u32(p_tile) + buf * Sh::kPBytes;
        if (fresh) {
          const uint32_t to = p_addr + (key >> 6) * (Sh::kN16 * 128) + (key & 7) * 2;
#pragma unroll
          for (int k = 0; k < RH; ++k) {
            const int r = wg * RH + k;
            st_u16(to + r * 128 + (((key & 63) >> 3 ^ (r & 7)) << 4), narrow(w[k], a.bf16));
          }
          if (wg < (Sh::kN16 - RT) / RH) {  // rows that the 16-bit product takes beyond the tile's: these rows' second parts
#pragma unroll
            for (int k = 0; k < RH; ++k) {
              const int r = RT + wg * RH + k;
              st_u16(to + r * 128 + (((key & 63) >> 3 ^ (r & 7)) << 4), 0);
            }
          }
        } else {
          // Weights of 11 bits (one rounding to fp16, exact in the parts but for their subnormal end): packed arithmetic.
          __half2 u[RH / 2];
#pragma unroll
          for (int k = 0; k < RH; k += 2) u[k / 2] = __floats2half2_rn(w[k] * vs, w[k + 1] * vs);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t code[RH / 2];
#pragma unroll
            for (int k = 0; k < RH / 2; ++k) {
              code[k] = sv::f8_pair_e4m3(u[k]);
              if (g < 3) u[k] = __hmul2(__hsub2(u[k], sv::f8_halves_e4m3(code[k])), __float2half2_rn(32.f));
            }
            const int n = g * RT + wg * RH;
            const uint32_t to = p_addr + (n >> 4) * (kBlock * 16) + key * 16 + (n & 15);
            if (RH == 8) st_v2(to, code[0] | code[1] << 16, code[RH / 2 - 2] | code[RH / 2 - 1] << 16);
            else st_u32(to, code[0] | code[1] << 16);
          }
        }
        sv::fence_proxy_async_smem();
        sv::tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) sv::mbar_arrive(&sh.p_full[buf]);
      }

      // ---- end of the segment: normalise and write, or leave partial rows
#pragma unroll
      for (int k = 0; k < RH; ++k) {
        float t = sum[k];
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (lane == 0) rw.sum[quad][own0 + k] = t;
      }
      const bool used = team < nb;
      if (used) wait_done(team + (nb - 1 - team) / kTeams * kTeams);  // the team's last block
      if (kTeams == 1 && nb > 1) wait_done(nb - 2);                   // (so that no phase is passed over)
      meet(kAll, 32 * kSoftmaxWarps);  // every sum, and every mark of spoiled entries, is there
      const bool whole = nb == s.nb;
      const int slot = lo > 0 ? 0 : 1;  // (a piece that goes on from the CTA before, or one that others go on with)
      const long long base = static_cast<long long>(at.b) * a.S * a.heads + at.kvh * a.G;
      const long long part = (static_cast<long long>(cta) * 2 + slot) * kMaxRows;
      // A thread per row weighs the teams' sums.  The exponent of a sum goes into its reference, here and for the join:
      // sums of like size, and the largest reference is that of what counts most.
      if (team == 0 && key < RH) {
        const int r = wg * RH + key;
        float hi[kTeams], low[kTeams], unit[kTeams], all[kTeams], hi2 = -INFINITY, lo2 = 0.f, total = 0.f;
#pragma unroll
        for (int t = 0; t < kTeams; ++t) {
          const float4 st = rw.st[t * RT + r];
          all[t] = (rw.sum[0][t * RT + r] + rw.sum[1][t * RT + r]) + (rw.sum[2][t * RT + r] + rw.sum[3][t * RT + r]);
          const int e = all[t] > 0.f && all[t] < INFINITY ? ilog2(all[t]) : 0;
          hi[t] = st.y;
          low[t] = st.z + e;
          unit[t] = exp2f(static_cast<float>(-e));
          all[t] *= unit[t];
          if (all[t] != 0.f && !((hi[t] - hi2) + (low[t] - lo2) <= 0.f)) {
            hi2 = hi[t];
            lo2 = low[t];
          }
        }
        float w[kTeams];
#pragma unroll
        for (int t = 0; t < kTeams; ++t) {
          w[t] = all[t] == 0.f ? -1.f : kTeams == 1 ? 1.f : exp2_small((hi[t] - hi2) + (low[t] - lo2));
          if (all[t] != 0.f) total += all[t] * w[t];
        }
        const bool none = total == 0.f;
        const float inv = none ? 0.f : 1.f / total;
#pragma unroll
        for (int t = 0; t < kTeams; ++t) rw.done[t * RT + r] = w[t] < 0.f ? -1.f : inv * unit[t] * w[t];  // (-1: saw no key)
        if (r < rows) {
          if (!whole) a.part_ml[part + r] = make_float4(hi2, lo2, total, 0.f);
          else if (a.lse) a.lse[base + rw.out[r]] = none ? -INFINITY : (hi2 + (lo2 + log2f(total))) * kLn2;
        }
      }
      meet(kAll, 32 * kSoftmaxWarps);
      float* other = reinterpret_cast<float*>(p_tile);  // [RT][D] of the second team (the products with P are done)
      static_assert(kTeams == 1 || RT * D * 4 <= 2 * Sh::kPBytes, "room for a team's rows");
      float o[RH];
      if (used) {
        uint32_t o0[RH], o1[RH], o2[RH], o3[RH];
        sv::tmem_start(o_addr, o0);
        sv::tmem_start(o_addr + RT, o1);
        sv::tmem_start(o_addr + 2 * RT, o2);
        sv::tmem_start(o_addr + 3 * RT, o3);
        sv::tmem_wait_ld();
        sv::tmem_use(o0);
        sv::tmem_use(o1);
        sv::tmem_use(o2);
        sv::tmem_use(o3);
#pragma unroll
        for (int n = 0; n < RH; ++n) {
          const float f = rw.done[own0 + n];
          o[n] = fmaf(__uint_as_float(o3[n]), 1.f / 32768, __uint_as_float(o2[n]) * (1.f / 1024));
          o[n] += fmaf(__uint_as_float(o1[n]), 1.f / 32, __uint_as_float(o0[n]));
          o[n] = f < 0.f ? 0.f : o[n] * f;
        }
        if (team == 1 && key < D) {
#pragma unroll
          for (int n = 0; n < RH; ++n) other[(wg * RH + n) * D + key] = o[n];
        }
      }
      if (kTeams == 2 && nb > 1) meet(kAll, 32 * kSoftmaxWarps);
      if (team == 0 && key < D) {
        bool spoils = false;
        if (tails > 0)
          for (int w = 0; w < kMaxTree / 32; ++w) spoils |= rw.spoiled[w] != 0;
#pragma unroll
        for (int n = 0; n < RH; ++n) {
          const int r = wg * RH + n;
          if (r >= rows) continue;
          if (kTeams == 2 && nb > 1) o[n] += other[r * D + key];
          if (spoils) o[n] += spoiled_sum<D>(a, at.b, at.kvh, s.Lq, rw.tok[r], key, rw.spoiled,
                                             tree ? rw.anc[rw.tok[r] - tok0] : nullptr);
          if (whole) static_cast<uint16_t*>(a.out)[(base + rw.out[r]) * D + key] = static_cast<uint16_t>(narrow(o[n], a.bf16));
          else a.part_o[(part + r) * D + key] = o[n];
        }
      }
      if (!whole && lo == 0 && tid == 32 * kSoftmaxWarps - 1) {
        Cut cut;
        cut.active = 1;
        cut.last = sh.shares.owner(at.start + kItemUnits<RT> + s.nb - 1);
        cut.b = at.b;
        cut.rows = rows;
        cut.row0 = row0;
        cut.base = base;
        a.cuts[cta] = cut;
      }
      sv::tc_fence_before_sync();
      meet(kAll, 32 * kSoftmaxWarps);  // the state may be set for the next item
      loads += nb + tails;
      uses[0] += (nb + 1) / 2;
      uses[1] += nb / 2;
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
// join_split-th group of rows of the item whose first piece CTA c has; a warp
// takes a row.  Bound by two dependent loads (the record, then all the rest).
template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv8_join_kernel(const Args a) {
  constexpr int kE = D / 32, kWarps = kJoinThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sv::griddep_wait();
  sv::griddep_launch_dependents();
  const Cut cut = a.cuts[blockIdx.x];
  const int errors = a.ctrl[sv::kKvCollect];  // (the main kernel has set them all)
  const int first = blockIdx.x, rows = cut.active ? cut.rows : 0;
  for (int i = blockIdx.y * kWarps + warp; i < rows; i += a.join_split * kWarps) {
    if (errors && a.bad[cut.b]) break;
    auto place = [&](int p) { return (static_cast<long long>(p) * 2 + (p == first ? 1 : 0)) * kMaxRows + i; };
    float hi = -INFINITY, lo = 0.f, sum = 0.f, o[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = 0.f;
    for (int p0 = first; p0 <= cut.last; p0 += 32) {  // (one round for up to 32 pieces)
      float4 ml = make_float4(-INFINITY, 0.f, 0.f, 0.f);
      if (p0 + lane <= cut.last) ml = a.part_ml[place(p0 + lane)];
      if (ml.z == 0.f) ml.x = -INFINITY;  // it saw no key
      // the piece that counts most, of those so far as well; what is not a number takes no part
      const float key = fmaxf(ml.x + ml.y, -INFINITY), old = sum == 0.f ? -INFINITY : fmaxf(hi + lo, -INFINITY);
      float most = key;
#pragma unroll
      for (int w = 16; w; w >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, w));
      float top = 0.f, low = 0.f;  // (nothing yet, or sums that are not a number)
      if (most > old) {
        const int from = __ffs(__ballot_sync(0xffffffffu, key == most)) - 1;
        top = __shfl_sync(0xffffffffu, ml.x, from);
        low = __shfl_sync(0xffffffffu, ml.y, from);
      } else if (old > -INFINITY) {
        top = hi;
        low = lo;
      }
      const float w = ml.z == 0.f ? 0.f : ml.z * exp2_small((ml.x - top) + (ml.y - low));
      const float held = sum == 0.f ? 0.f : exp2_small((hi - top) + (lo - low));
      sum *= held;
#pragma unroll
      for (int e = 0; e < kE; ++e) o[e] *= held;
      hi = top;
      lo = low;
      const int n = min(32, cut.last - p0 + 1);
#pragma unroll 4
      for (int p = 0; p < n; ++p) {
        const float f = __shfl_sync(0xffffffffu, w, p);
        const float* from = a.part_o + place(p0 + p) * D + lane * kE;
        float x[kE];
#pragma unroll
        for (int e = 0; e < kE; e += 2) {
          const float2 v = *reinterpret_cast<const float2*>(from + e);
          x[e] = v.x;
          x[e + 1] = v.y;
        }
        sum += f;
        if (f != 0.f) {
#pragma unroll
          for (int e = 0; e < kE; ++e) o[e] = fmaf(f, x[e], o[e]);
        } else {  // a weight that underflows: only what is not finite counts
#pragma unroll
          for (int e = 0; e < kE; ++e)
            if (!isfinite(x[e])) o[e] += x[e];
        }
      }
    }
    const bool none = sum == 0.f;
    const float inv = none ? 0.f : 1.f / sum;
    const int tok = (cut.row0 + i) / a.G, g = (cut.row0 + i) - tok * a.G;
    const long long orow = cut.base + static_cast<long long>(tok) * a.heads + g;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + orow * D + lane * kE);
#pragma unroll
    for (int e = 0; e < kE; e += 2)
      dst[e / 2] = none ? 0u : narrow(o[e] * inv, a.bf16) | narrow(o[e + 1] * inv, a.bf16) << 16;
    if (a.lse && lane == 0) a.lse[orow] = none ? -INFINITY : (hi + (lo + log2f(sum))) * kLn2;
  }
  if (errors == 0) {  // (the same answer in every CTA)
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.ctrl[sv::kKvErr] = 0;
    return;
  }
  for (int b = blockIdx.x * a.join_split + blockIdx.y; b < a.B; b += gridDim.x * a.join_split) {
    if (!a.bad[b]) continue;
    const int n = a.q_len ? a.q_len[b] : a.S;
    const long long count = static_cast<long long>(n < 0 || n > a.S ? a.S : n) * a.heads;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + static_cast<long long>(b) * a.S * a.heads * D);
    for (long long i = threadIdx.x; i < count * D / 8; i += kJoinThreads) dst[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (long long i = threadIdx.x; i < count; i += kJoinThreads)
        a.lse[static_cast<long long>(b) * a.S * a.heads + i] = -INFINITY;
  }
  // the last CTA leaves the marks ready for the next call
  __shared__ int s_last;
  __syncthreads();
  if (threadIdx.x == 0) s_last = sv::kv_last_cta(a.ctrl);
  __syncthreads();
  if (!s_last) return;
  for (int b = threadIdx.x; b < a.B; b += kJoinThreads) a.bad[b] = 0;
  __syncthreads();
  if (threadIdx.x == 0) sv::kv_publish(a.ctrl);
}

// --------------------------------------------------------------------- host
bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

bool dims_ok(const spec_kv8_attn_dims& d) {
  return (d.head_dim == 64 || d.head_dim == 128) && d.kv_heads >= 1 && d.heads >= d.kv_heads && d.heads <= 1024 &&
         d.heads % d.kv_heads == 0 && d.heads / d.kv_heads <= 64 &&
         (d.dtype == SPEC_ATTN_BF16 || d.dtype == SPEC_ATTN_FP16) &&
         (d.format == SPEC_KV8_E4M3 || d.format == SPEC_KV8_E5M2) && d.B >= 1 && d.B <= kMaxBatch && d.S >= 1 &&
         d.S <= 256 && static_cast<int64_t>(d.B) * d.S <= (1 << 24) && d.page_size >= 1 && d.num_pages >= 1 &&
         d.max_pages >= 1 && static_cast<int64_t>(d.max_pages) * d.page_size < (1ll << 31) &&
         static_cast<int64_t>(d.num_pages) * d.page_size < (1ll << 31) && d.q_stride % 8 == 0 &&
         d.q_stride >= static_cast<int64_t>(d.heads) * d.head_dim && d.q_stride <= (1ll << 31);
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
  size_t bad, cuts, part_ml, part_o, total;
};

// What a call expects to be zero and leaves so (the control words and the marks) lies in front and takes the same
// bytes for every call; what is behind it is written before it is read.
Layout layout(int head_dim) {
  Layout l;
  const size_t rows = static_cast<size_t>(kMaxGrid) * 2 * kMaxRows;
  l.bad = sv::kKvCtrlBytes;
  l.cuts = l.bad + up(4 * static_cast<size_t>(kMaxBatch));
  l.part_ml = l.cuts + up(sizeof(Cut) * kMaxGrid);
  l.part_o = l.part_ml + up(sizeof(float4) * rows);
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

// A tensor of `rank` dimensions (strides in bytes from the second on) with rows of row_bytes as the swizzle; zeros outside.
bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, int row_bytes) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t step[5] = {1, 1, 1, 1, 1};
  return fn(map, type, rank, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The pool as [heads][groups of eight rows][key, value][eight rows][head_dim]: a box of rows comes with its keys and
// values by turns, eight rows each.
bool encode_pool(CUtensorMap* map, const void* pool, int head_dim, int kv_heads, int64_t rows, int box) {
  const cuuint64_t D = head_dim, H = kv_heads, entry = 2 * H * D;
  const cuuint64_t dims[5] = {D, 8, 2, static_cast<cuuint64_t>((rows + 7) / 8), H};
  const cuuint64_t strides[4] = {entry, H * D, 8 * entry, D};
  const cuuint32_t boxes[5] = {static_cast<cuuint32_t>(D), 8, 2, static_cast<cuuint32_t>(box / 8), 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, pool, 5, dims, strides, boxes, head_dim);
}

// Staged entries: boxes of 64 columns of one head of `box` tokens.
bool encode_staged(CUtensorMap* map, bool bf16, const void* staged, int head_dim, int kv_heads, int64_t tokens, int box) {
  const cuuint64_t D = head_dim, H2 = 2 * static_cast<cuuint64_t>(kv_heads);
  const cuuint64_t dims[3] = {D, H2, static_cast<cuuint64_t>(tokens)}, strides[2] = {2 * D, 2 * H2 * D};
  const cuuint32_t boxes[3] = {64, 1, static_cast<cuuint32_t>(box)};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, staged, 3, dims, strides,
                boxes, 128);
}

template <int D, int RT>
spec_status launch(const Args& a, const CUtensorMap (&maps)[2], const sv::DeviceInfo& dev, cudaStream_t s) {
  using Sh = Shape<D, RT>;
  constexpr size_t kBytes = 1024 + Sh::kSlots * Sh::kSlotBytes + 2 * Sh::kPBytes + Sh::kQBytes + Sh::kQ16Bytes +
                            (sizeof(Sync) + 15) / 16 * 16 + sizeof(Rows<RT, Sh::kTeams, Sh::kSlots>);
  static_assert(kBytes <= 232448, "shared memory of one CTA");
  static_assert(kBytes > 116 * 1024, "one CTA per SM: the grid is as many as there are");
  static_assert(Sh::kSlots >= 4 && Sh::kSlots <= kMaxSlots, "two blocks of 16-bit entries take four slots");
  static_assert(Sh::kPBytes % 1024 == 0 && Sh::kQBytes % 1024 == 0 && Sh::kQ16Bytes % 1024 == 0, "tiles start on 1024 bytes");
  static bool done[64] = {false};
  if (!done[dev.device]) {
    if (cudaFuncSetAttribute(kv8_attn_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kBytes)) != cudaSuccess)
      return SPEC_ERR_CUDA;
    done[dev.device] = true;
  }
  const int grid = dev.sm_count < kMaxGrid ? dev.sm_count : kMaxGrid;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Sh::kThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kv8_attn_kernel<D, RT>, a, maps[0], maps[1]) != cudaSuccess) return SPEC_ERR_CUDA;
  if (sv::launch_dependent(kv8_join_kernel<D>, dim3(grid, a.join_split), dim3(kJoinThreads), s, a) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

// The smallest tile that holds a token's rows of a group, or an even share of them where even the largest does not.
template <int D>
spec_status launch(Args& a, const CUtensorMap (&maps)[2], const sv::DeviceInfo& dev, cudaStream_t s) {
  const int rows = a.S * a.G, tiles = (rows + kMaxRows - 1) / kMaxRows, each = ((rows + tiles - 1) / tiles + 7) / 8 * 8;
  a.tile_rows = each;
  if (each <= 8) return launch<D, 8>(a, maps, dev, s);
  if (each <= 16) return launch<D, 16>(a, maps, dev, s);
  if (each <= 32) return launch<D, 32>(a, maps, dev, s);
  if (each <= 40) return launch<D, 40>(a, maps, dev, s);
  return launch<D, 48>(a, maps, dev, s);
}

}  // namespace

extern "C" {

size_t spec_kv8_attention_workspace_bytes(spec_kv8_attn_dims dims) {
  return dims_ok(dims) ? layout(dims.head_dim).total : 0;
}

spec_status spec_kv8_attention(const void* q, const void* pool, const float* scales, const int32_t* block_table,
                               const int32_t* seq_len, const void* staged, const int32_t* parents,
                               const int32_t* q_len, float scale, void* out, float* out_lse, spec_kv8_attn_dims dims,
                               void* workspace, size_t workspace_bytes, spec_stream_t stream) {
  if (!q || !pool || !scales || !block_table || !seq_len || !staged || !out || !workspace) return SPEC_ERR_ARG;
  if (!(scale > 0.f && scale <= 65536.f)) return SPEC_ERR_ARG;
  if (!dims_ok(dims)) return SPEC_ERR_DIMS;
  if (misaligned(q, 16) || misaligned(pool, 16) || misaligned(staged, 16) || misaligned(out, 16) ||
      misaligned(workspace, 16) || misaligned(scales, 4) || misaligned(block_table, 4) || misaligned(seq_len, 4) ||
      misaligned(parents, 4) || misaligned(q_len, 4) || misaligned(out_lse, 4))
    return SPEC_ERR_ALIGN;
  if (workspace_bytes < spec_kv8_attention_workspace_bytes(dims)) return SPEC_ERR_WORKSPACE;
  sv::DeviceInfo dev;
  const int st = sv::current_device(dev);
  if (st != SPEC_OK) return static_cast<spec_status>(st);
  Args a = {};
  a.q = q;
  a.staged = staged;
  a.pool = static_cast<const uint8_t*>(pool);
  a.scales = scales;
  a.bt = block_table;
  a.len = seq_len;
  a.q_len = q_len;
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
  a.format = dims.format;
  a.bf16 = dims.dtype == SPEC_ATTN_BF16;
  a.q_stride = dims.q_stride;
  // division by the page size, exact for positions below 2^31
  int log = 0;
  while ((1ll << log) < dims.page_size) ++log;
  a.page_mul = static_cast<uint32_t>((1ull << (31 + log)) / static_cast<uint64_t>(dims.page_size) + 1);
  a.page_shift = 31 + log;
  // the largest boxes that pages and blocks divide into; below eight rows (the swizzle's unit) row by row
  a.box = kBlock;
  while (a.box >= 8 && dims.page_size % a.box != 0) a.box /= 2;
  if (a.box < 8) a.box = 0;
  const int rows = dims.S * a.G;
  a.least = rows <= 16 ? 1 : 3;
  a.join_split = rows <= 8 ? 1 : (rows < 48 ? (rows + 7) / 8 : 6);
  const Layout l = layout(dims.head_dim);
  char* ws = static_cast<char*>(workspace);
  a.ctrl = reinterpret_cast<int*>(ws);
  a.bad = reinterpret_cast<int*>(ws + l.bad);
  a.cuts = reinterpret_cast<Cut*>(ws + l.cuts);
  a.part_ml = reinterpret_cast<float4*>(ws + l.part_ml);
  a.part_o = reinterpret_cast<float*>(ws + l.part_o);
  a.fresh_box = dims.S < kBlock ? (dims.S + 7) / 8 * 8 : kBlock;  // (rows behind are zeroed or not looked at)
  CUtensorMap maps[2] = {};
  const int64_t tokens = static_cast<int64_t>(dims.B) * dims.S;
  // (without boxes the pool's map is not used)
  if ((a.box && !encode_pool(&maps[0], pool, dims.head_dim, dims.kv_heads,
                             static_cast<int64_t>(dims.num_pages) * dims.page_size, a.box)) ||
      !encode_staged(&maps[1], a.bf16, staged, dims.head_dim, dims.kv_heads, tokens, a.fresh_box))
    return SPEC_ERR_CUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dims.head_dim == 64 ? launch<64>(a, maps, dev, s) : launch<128>(a, maps, dev, s);
}

}  // extern "C"
