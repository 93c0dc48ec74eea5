// Attention of new tokens over a paged bf16 cache (sm_103a).
//
// Sequence b has n_b new tokens, rows query_start[b] .. query_start[b + 1] - 1 of q, and L_b keys; its token i sits at
// position p = L_b - n_b + i.  For query head h of key head h / G (G = H / Hkv), over the visible keys j (j < L_b, with
// `causal` j <= p, with a window j > p - window):
//   s_j = scale q . k_j,  out = sum_j e^(s_j - m) v_j / (sum_j e^(s_j - m) + e^(sink - m)),  lse = ln of the denominator.
//
// Rows and tiles.  The G query heads of a key head share its keys, so row r of a (sequence, key head) is head r % G of
// token r / G, and an item is a block of its rows: 256 (two row tiles of 128) or, where sequences bring few rows, 128.
// Keys come in tiles of 128.  Items lie end to end on a line, each as long as the key tiles that its rows see; the line
// is cut into equal slices, one per CTA (one CTA per SM).  So a decode batch of any lengths, one long row or a causal
// prompt load every SM alike.  An item cut by a slice's end leaves its parts (unnormalised sums, maximum, denominator)
// in the workspace, and combine_kernel adds them in order: results do not depend on timing.
//
// In a CTA, two streams alternate on the tensor cores: while one's softmax runs, the other's products do.  With two row
// tiles each is a stream, and both use every key tile; with one, the streams take the even and the odd key tiles with
// sums of their own, joined at the item's end.
//   S_t = Q_t K^T        128 x 64, half a key tile at a time, both operands from shared memory
//   P_t = 2^(S c - m)    by the stream's four softmax warps, a row per thread: fp32 statistics, P rounded to bf16 and
//                        written over S in tensor memory; the maximum moves only when a half tile exceeds it by more
//                        than 8 in base 2 (P <= 2^8 loses nothing in bf16), and only then are the sums O_t rescaled
//   O_t += P_t V         A from tensor memory, V as stored (dims contiguous)
// S_t has two buffers: the next half tile's scores are made while the softmax of this one runs, so that neither waits for
// the other (with one buffer of a whole key tile per stream a tile of 256 rows took 4350 cycles).
// The denominator sums the unrounded weights: P's rounding (2^-9 of each weight on average, as often up as down) then
// touches the output as the output's own rounding does, and the lse not at all.
//
// Warps: 0-3 and 4-7 softmax, 8-11 bring keys and values (32 rows of each tile per warp) by tensor copies, 12 and 13
// issue a stream's products each, 14 and 15 bring the queries and look through the values of tiles that some row sees in
// part.  Where the page size is a multiple of 8, a copy's box is as many rows as divide both a page and a tile; other
// pages are gathered row by row, four to a copy.  What no row of the item sees is asked for past the tensor's end, which
// reads as zeros.  Tensor memory: S_t 2 x 2 x 64 columns, O_t 2 x 128.
//
// Measured (64 query heads, 8 key heads of 128), calls in a captured graph: a prompt of 8192 tokens 734 us = 1.5 PFLOP/s in a
// burst of 24 (741 on another GPU), 789 us on and on at the power limit (1942 MHz).  Four fifths of that are the
// softmax's latency (1250 cycles per half tile and stream, 2800 a key tile; the products need 2560), the rest passes
// between items and in their parts; of a 4096-token prompt's 220 us it is two thirds.  64 single tokens over contexts up to
// 32K 637 us, the rate of a copy; one token over 4096 keys 13.0 us, nearly all of it latency.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "launch.h"

namespace dsa {
namespace {

constexpr int kKeys = 128;                   // keys per tile
constexpr int kThreads = 512;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.0f;                // base-2 headroom before the running maximum moves
constexpr int kPlanMax = 512;                // row blocks (and sequences) that a CTA plans by itself
constexpr int kItemCost = 3;                 // an item's fixed cost, in key tiles (8192-token prompt: 2 748, 3 741, 4 747 us)

// n / d for 0 <= n < 2^31 as a product and a shift (Granlund and Montgomery: with 2^(s-1) < d <= 2^s and mul =
// ceil(2^(31+s) / d) the excess mul d - 2^(31+s) < 2^s is too small to reach the next quotient).  Every role finds its
// way through the items with half a dozen of them, one after the other.
struct Divisor {
  uint32_t mul;
  int shift;
  __device__ __forceinline__ int of(int n) const { return (int)(((uint64_t)(uint32_t)n * mul) >> shift); }
};

struct AttnArgs {
  const uint16_t* q;
  int64_t ldq;
  const int32_t* start;        // [B + 1]
  const int32_t* lens;         // [B]
  const int32_t* table;        // [B, bt_stride]
  int64_t bt_stride;
  const uint16_t* v;           // (keys come by copies alone)
  int64_t num_blocks, block_stride, row_stride, head_stride;
  int block_rows, head_rows;   // block_stride and head_stride in rows of the copies' tensor
  int head_cols;               // and what of head_stride lies within a row, in elements
  int no_row;                  // the tensor's rows: one past its end
  int box;                     // rows of a copy: 8 .. 128 dividing page and tile, or 1 (gathered)
  int q_boxes;                 // G divides 128: a row tile of queries is one box of tokens and heads
  int64_t cap;                 // keys a block-table row can hold
  int block_size;
  int64_t T;
  int B, H, Hkv, G;
  Divisor by_group, by_block;  // by G and by block_size
  int causal, window;          // window 0: none
  float scale_log2;            // softmax scale in base 2
  const float* sink;           // nullable
  uint16_t* out;
  int64_t ldo;
  float* lse;                  // nullable
  // workspace
  int32_t* meta;               // [1 + CTAs][12]
  float* ml;                   // [2 * CTAs][rows][2]
  float* part;                 // [2 * CTAs][rows][D]
  int64_t* prefix;             // the plan, where it is not made in shared memory
  int32_t* first;
  int32_t* seq;
  int planned;
  int limit;                   // row blocks there can be: sequences that overlap would bring more
};

// ------------------------------------------------------------------ items
struct Seq {
  int s, n, L;                 // first row of q, new tokens, keys
};

// What the arguments say of sequence b, or an empty one (`bad`) where that is no range of the T rows.
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b, bool& bad) {
  Seq q;
  q.s = a.start[b];
  const int64_t e = a.start[b + 1];
  q.L = a.lens[b];
  q.n = (int)(e - q.s);
  if (q.s < 0 || e < q.s || e > a.T) {
    bad = true;
    q.n = 0;
  }
  if (q.L < 0) {
    bad = true;
    q.L = 0;
  }
  return q;
}

struct Item {
  int b, s, n, L;
  int row0, rows;              // rows row0 .. row0 + rows - 1 of the (sequence, key head)
  int lo, hi;                  // keys that some row sees
  int tile0, tiles;            // key tiles of [lo, hi)
};

// Visible keys of the token at position p, as [lo, hi).
__device__ __forceinline__ int low_key(const AttnArgs& a, int p) {
  return a.window > 0 ? (int)max((int64_t)p - a.window + 1, (int64_t)0) : 0;
}
__device__ __forceinline__ int high_key(const AttnArgs& a, int L, int p) {
  const int hi = a.causal ? max(0, min(L, p + 1)) : L;
  return (int)min((int64_t)hi, a.cap);
}

template <int kRows>
__device__ __forceinline__ Item make_item(const AttnArgs& a, const Seq& q, int b, int block) {
  Item it;
  it.b = b, it.s = q.s, it.n = q.n, it.L = q.L;
  it.row0 = block * kRows;
  it.rows = min(kRows, q.n * a.G - it.row0);
  const int i0 = a.by_group.of(it.row0), i1 = a.by_group.of(it.row0 + it.rows - 1);
  it.lo = low_key(a, q.L - q.n + i0);
  it.hi = high_key(a, q.L, q.L - q.n + i1);
  it.tile0 = it.lo / kKeys;
  it.tiles = it.hi > it.lo ? (it.hi - 1) / kKeys - it.tile0 + 1 : 0;
  return it;
}

// Exclusive prefix sum over the NT threads of the block; returns the sum of the threads before, `total` of all.
template <int NT, typename V>
__device__ __forceinline__ V block_scan(V v, int64_t* scratch, V& total) {
  V* warp_s = reinterpret_cast<V*>(scratch);
  const int lane = (int)threadIdx.x & 31, w = (int)threadIdx.x >> 5;
  V incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_s[w] = incl;
  __syncthreads();
  V before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    const V c = warp_s[i];
    if (i < w) before += c;
    all += c;
  }
  __syncthreads();
  total = all;
  return before + incl - v;
}

// The plan: first[b] = row blocks of the sequences before b; for row block e of sequence seq[e], prefix[e] = the length
// of the row blocks before it, each kItemCost and its key tiles (at least one, so that a block that sees nothing still
// has its turn).  A row block has an item per key head; these lie side by side on the line, whose length is
// prefix[count] * Hkv.
// V is wide enough for the line: 32 bits where a CTA plans (at most kPlanMax row blocks of at most 2^22 key tiles).
template <int kRows, int NT, typename V>
__device__ int make_plan(const AttnArgs& a, V* prefix, int32_t* first, int32_t* seq, int64_t* scratch, bool tell) {
  int64_t many = 0;
  bool bad = false;
  for (int b0 = 0; b0 < a.B; b0 += NT) {
    const int b = b0 + (int)threadIdx.x;
    int64_t c = 0;
    if (b < a.B) c = ((int64_t)sequence(a, b, bad).n * a.G + kRows - 1) / kRows;
    // (more than there can be counts as one more: then the sequences overlap)
    V total;
    const V before = block_scan<NT, V>((V)min(c, (int64_t)a.limit + 1), scratch, total);
    if (b < a.B) first[b] = (int32_t)min(many + (int64_t)before, (int64_t)INT32_MAX);
    many = min(many + (int64_t)total, (int64_t)1 << 40);
  }
  __syncthreads();
  const int count = (int)min(many, (int64_t)a.limit);
  if (many > a.limit) bad = true;
  V carry = 0;
  for (int e0 = 0; e0 < count; e0 += NT) {
    const int e = e0 + (int)threadIdx.x;
    V c = 0;
    if (e < count) {
      int lo = 0, hi = a.B;                        // the last sequence with first[b] <= e
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= e) lo = mid;
        else hi = mid;
      }
      seq[e] = lo;
      const Seq q = sequence(a, lo, bad);
      const Item it = make_item<kRows>(a, q, lo, e - first[lo]);
      c = (V)(kItemCost + max(it.tiles, 1));
      if (it.L > a.cap) bad = true;                // keys past the block table's row
    }
    V total;
    const V before = block_scan<NT, V>(c, scratch, total);
    if (e < count) prefix[e] = carry + before;
    carry += total;
  }
  if (threadIdx.x == 0) prefix[count] = carry;
  if (tell && bad) raise_error(DSA_DEVERR_INDEX);
  __syncthreads();
  return count;
}

// The same plan for at most 32 sequences of few row blocks by one warp, a sequence and then a row block per lane: one trip
// to memory and no barrier but the last.  One token over 4096 keys 12.8 us, by all warps 13.3; 32 x 2 tokens 23.7 and 24.4;
// with 58 and more row blocks no difference.
constexpr int kWarpPlan = 96;
template <int kRows>
__device__ int make_small_plan(const AttnArgs& a, uint32_t* prefix, int32_t* first, int32_t* seq, int* count_s, bool tell) {
  if (threadIdx.x < 32) {
    const int lane = (int)threadIdx.x;
    bool bad = false;
    Seq q{0, 0, 0};
    if (lane < a.B) q = sequence(a, lane, bad);
    const uint32_t c = (uint32_t)min(((int64_t)q.n * a.G + kRows - 1) / kRows, (int64_t)a.limit + 1);
    uint32_t incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t mine = incl - c, all = __shfl_sync(0xFFFFFFFFu, incl, 31);
    if (lane < a.B) first[lane] = (int32_t)mine;
    if (all > (uint32_t)a.limit) bad = true;
    const int count = (int)min(all, (uint32_t)a.limit);
    uint32_t carry = 0;
    for (int e0 = 0; e0 < count; e0 += 32) {
      const int e = e0 + lane;
      int b = 0;                                   // the last sequence that begins at or before row block e
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint32_t f = __shfl_sync(0xFFFFFFFFu, mine, (b + o) & 31);
        if (b + o < a.B && f <= (uint32_t)e) b += o;
      }
      Seq s;
      s.s = __shfl_sync(0xFFFFFFFFu, q.s, b), s.n = __shfl_sync(0xFFFFFFFFu, q.n, b), s.L = __shfl_sync(0xFFFFFFFFu, q.L, b);
      const uint32_t f = __shfl_sync(0xFFFFFFFFu, mine, b);
      uint32_t v = 0;
      if (e < count) {
        seq[e] = b;
        const Item it = make_item<kRows>(a, s, b, e - (int)f);
        v = (uint32_t)(kItemCost + max(it.tiles, 1));
        if (it.L > a.cap) bad = true;
      }
      uint32_t sum = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += y;
      }
      if (e < count) prefix[e] = carry + sum - v;
      carry += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (lane == 0) {
      prefix[count] = carry;
      *count_s = count;
    }
    if (tell && bad) raise_error(DSA_DEVERR_INDEX);
  }
  __syncthreads();
  return *count_s;
}

template <int kRows>
__global__ void __launch_bounds__(1024) plan_kernel(const AttnArgs a) {
  __shared__ int64_t warp_s[32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int count = make_plan<kRows, 1024, int64_t>(a, a.prefix, a.first, a.seq, warp_s, true);
  if (threadIdx.x == 0) a.meta[7] = count;
}

// One CTA's pieces of the line, in order.
struct Pieces {
  const uint32_t* plan_s;      // the CTA's own plan: prefix, first, seq (kPlanMax + 8, kPlanMax, kPlanMax)
  int e;
  int64_t x, end;

  __device__ __forceinline__ int64_t prefix(const AttnArgs& a, int i) const { return a.planned ? a.prefix[i] : (int64_t)plan_s[i]; }
  __device__ __forceinline__ int first(const AttnArgs& a, int b) const {
    return a.planned ? a.first[b] : (int)plan_s[kPlanMax + 8 + b];
  }
  __device__ __forceinline__ int seq(const AttnArgs& a, int i) const {
    return a.planned ? a.seq[i] : (int)plan_s[2 * kPlanMax + 8 + i];
  }

  __device__ __forceinline__ void begin(const AttnArgs& a, int count, int64_t from, int64_t to) {
    x = from, end = to;
    int lo = 0, hi = count;
    while (hi - lo > 1) {                          // the row block that holds x
      const int mid = (lo + hi) >> 1;
      if (prefix(a, mid) * a.Hkv <= x) lo = mid;
      else hi = mid;
    }
    e = lo;
  }
};

struct Piece {
  Item it;
  int hk;                      // key head
  int t0, len, cost;           // key tiles t0 .. t0 + len - 1 of the item's `cost`
  int block = -1;              // the row block that `it` describes (that of several key heads in a row)
};

template <int kRows>
__device__ __forceinline__ bool next_piece(const AttnArgs& a, Pieces& ps, Piece& p) {
  while (ps.x < ps.end) {
    const int64_t base = ps.prefix(a, ps.e);
    const int length = (int)(ps.prefix(a, ps.e + 1) - base);
    const int64_t rem = ps.x - base * a.Hkv;
    if (a.Hkv <= 128) p.hk = (int)((uint32_t)rem / (uint32_t)length);      // length <= 2^24 + kItemCost
    else p.hk = (int)(rem / length);
    const int from = (int)(rem - (int64_t)p.hk * length), to = (int)min((int64_t)length, from + (ps.end - ps.x));
    p.cost = length - kItemCost;
    p.t0 = max(from - kItemCost, 0);
    p.len = max(to - kItemCost, 0) - p.t0;
    const int e = ps.e;
    ps.x += to - from;
    if (p.hk == a.Hkv - 1 && to == length) ++ps.e;
    if (p.len == 0) continue;                      // the slice ends within the item's fixed cost
    if (e != p.block) {
      const int b = ps.seq(a, e);
      bool bad = false;
      p.it = make_item<kRows>(a, sequence(a, b, bad), b, e - ps.first(a, b));
      p.block = e;
    }
    return true;
  }
  return false;
}

// The key tiles that every row of the item sees whole are those of [from, to).  In the others, a value that some row
// must not see would be a factor of its zero weight.
struct Whole {
  int from, to;
  __device__ __forceinline__ bool has(int tile) const { return tile >= from && tile < to; }
};
__device__ __forceinline__ Whole whole_tiles(const AttnArgs& a, const Item& it) {
  const int i0 = a.by_group.of(it.row0), i1 = a.by_group.of(it.row0 + it.rows - 1);
  const int least_hi = high_key(a, it.L, it.L - it.n + i0), most_lo = low_key(a, it.L - it.n + i1);
  return {(int)(((int64_t)most_lo + kKeys - 1) / kKeys), least_hi / kKeys};
}

// ------------------------------------------------------------------ tensor memory and barriers
// Shared-memory descriptors (128-byte swizzle) in two words: the high one holds the stride of 8-row groups (1024 bytes),
// the version and the swizzle; the low one the address and the stride of 64-element blocks, which only V's tiles use
// (dims contiguous).  Steps within a tile are additions to the low word.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t block) { return (addr >> 4) | (block >> 4) << 16; }

// One thread of the warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

// D (+)= A B, both from shared memory.
template <bool kAdd>
__device__ __forceinline__ void mma_ss(uint32_t tmem_d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n mov.b64 da, {%1, %3};\n mov.b64 db, {%2, %3};\n setp.ne.b32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n}" ::"r"(tmem_d),
      "r"(a), "r"(b), "r"(kDescHigh), "r"(idesc), "n"(kAdd ? 1 : 0)
      : "memory");
}

// D (+)= A B with A [128 rows][16 elements] in tensor memory: row r in lane r, elements 2c and 2c + 1 in column c.
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 db;\n mov.b64 db, {%2, %3};\n setp.ne.b32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n}" ::"r"(tmem_d),
      "r"(tmem_a), "r"(b), "r"(kDescHigh), "r"(idesc), "r"(add)
      : "memory");
}

// Consecutive 32-bit columns of the thread's own lane: load (complete on return) and store (complete at the wait).
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "{\n tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n tcgen05.wait::ld.sync.aligned;\n}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
               : "memory");
}

__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[64]) {
  tmem_ld64_issue(taddr, r);
  tmem_ld64_wait(r);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations at once.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Named barrier over n threads that also tells whether all of them are well.
__device__ __forceinline__ bool all_well(int bar, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n bar.red.and.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(bar), "r"(n), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// Four rows of 64 elements, 128 bytes each, at (x, y0 .. y3) into neighbouring rows of shared memory.
__device__ __forceinline__ void gather4(uint32_t dst, const void* tmap, uint32_t bar, int x, const int (&y)[4]) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
      : "memory");
}

// Box at (x, y, z) of a tensor of three dimensions.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("{\n .reg .b64 st;\n mbarrier.arrive.shared::cta.b64 st, [%0], %1;\n}" ::"r"(bar), "r"(n) : "memory");
}

// 16 bytes, or zeros where there is nothing to copy (then src is not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Bits [lo, hi) of a word, for any lo and hi.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  const int l = min(max(lo, 0), 32), h = min(max(hi, 0), 32);
  const uint32_t below_h = h >= 32 ? ~0u : (1u << h) - 1u, below_l = l >= 32 ? ~0u : (1u << l) - 1u;
  return below_h & ~below_l;
}

template <int D, int kTiles>
struct Shape {
  static constexpr int kRows = 128 * kTiles;
  static constexpr uint32_t kTile = 128u * D * 2u;                  // a tile of Q, K or V
  static constexpr int kStages = (D == 128 ? 4 : 8) + (kTiles == 1 ? 1 : 0) - (D == 64 ? 1 : 0);
  static constexpr uint32_t kStageOff = kTiles * kTile;
  static constexpr uint32_t kPlanOff = kStageOff + kStages * kTile;          // prefix, first, seq
  static constexpr uint32_t kMaskOff = kPlanOff + 4 * (kPlanMax + 8) + 4 * kPlanMax * 2;  // keys that exist [8][4] words
  static constexpr uint32_t kBadOff = kMaskOff + 8 * 16;            // values that are no numbers, per piece [16]
  static constexpr uint32_t kOutOff = kBadOff + 64;                 // results on their way out, 2 KB per softmax warp
  static constexpr uint32_t kStatOff = kOutOff + 8 * 2048;          // (m, l) [stream][128]
  static constexpr uint32_t kBarOff = kStatOff + 2048;
  static constexpr int kBars = 2 * kStages + 2 * 8 + 8 + 2;
  static constexpr uint32_t kCtlOff = kBarOff + 8 * 48;             // abort, TMEM base
  static constexpr uint32_t kScanOff = kCtlOff + 16;
  static constexpr size_t kSmem = 1024 + kScanOff + kThreads / 32 * 8;
  static_assert(kBars <= 48 && kStages <= 8 && kSmem <= 232448, "shared memory");
};

template <int D, int kTiles>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                                                              const __grid_constant__ CUtensorMap tmv,
                                                              const __grid_constant__ AttnArgs a) {
  using Sh = Shape<D, kTiles>;
  constexpr int kStages = Sh::kStages, kRows = Sh::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sm32 = smem_u32(sm);
  uint32_t* prefix_s = reinterpret_cast<uint32_t*>(sm + Sh::kPlanOff);
  int32_t* first_s = reinterpret_cast<int32_t*>(prefix_s + kPlanMax + 8);
  int32_t* seq_s = first_s + kPlanMax;
  uint32_t* mask_s = reinterpret_cast<uint32_t*>(sm + Sh::kMaskOff);
  volatile int* bad_s = reinterpret_cast<volatile int*>(sm + Sh::kBadOff);
  float2* stat_s = reinterpret_cast<float2*>(sm + Sh::kStatOff);
  int* ctl = reinterpret_cast<int*>(sm + Sh::kCtlOff);
  volatile int* abort_flag = ctl;
  const uint32_t bars = sm32 + Sh::kBarOff;
  // barrier numbers: stages full, stages empty, then per stream, then a ring of the tiles that are looked through
  constexpr int kFull = 0, kEmpty = kStages, kQFull = 2 * kStages, kQFree = kQFull + 2, kSFull = kQFree + 2,
                kPFull = kSFull + 4, kODone = kPFull + 4, kLook = kODone + 4, kDrain = kLook + 8;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };

  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const unsigned long long limit = wait_limit_ns();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(kFull + i), 4);
      mbar_init(bar(kEmpty + i), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kQFull + t), a.q_boxes ? 1 : 64);
      mbar_init(bar(kQFree + t), kTiles == 2 ? 1 : 2);
      for (int h = 0; h < 2; ++h) {
        mbar_init(bar(kSFull + 2 * t + h), 1);
        mbar_init(bar(kPFull + 2 * t + h), 4);
        mbar_init(bar(kODone + 2 * t + h), 1);
      }
    }
    for (int i = 0; i < 8; ++i) mbar_init(bar(kLook + i), 4);
    mbar_init(bar(kDrain), 1);
    mbar_init(bar(kDrain + 1), 1);
    ctl[0] = 0;
    if (a.q_boxes) tma_prefetch_desc(&tmq);
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) tmem_alloc(smem_u32(ctl + 1), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)ctl[1];
  grid_launch_dependents();
  grid_dependency_wait();

  // the plan, and this CTA's slice of the line
  Pieces ps;
  ps.plan_s = prefix_s;
  int count;
  if (a.planned) {
    count = *reinterpret_cast<volatile int32_t*>(a.meta + 7);
  } else if (a.B <= 32 && a.limit <= kWarpPlan) {
    count = make_small_plan<kRows>(a, prefix_s, first_s, seq_s, ctl + 2, blockIdx.x == 0);
  } else {
    count = make_plan<kRows, kThreads, uint32_t>(a, prefix_s, first_s, seq_s, reinterpret_cast<int64_t*>(sm + Sh::kScanOff), blockIdx.x == 0);
  }
  const int64_t C = gridDim.x;
  const int c = (int)blockIdx.x;
  const int64_t line = count > 0 ? ps.prefix(a, count) * a.Hkv : 0;
  if (line < (1 << 22)) ps.begin(a, count, (uint32_t)line * (uint32_t)c / (uint32_t)C, (uint32_t)line * (uint32_t)(c + 1) / (uint32_t)C);
  else ps.begin(a, count, line * c / C, line * (c + 1) / C);      // (a 64-bit division takes several times as long)

  if (warp < 8) {
    // ================================ softmax ================================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    const int t = warp >> 2;                       // stream
    const int r = 32 * (warp & 3) + lane;          // row in its tile = TMEM lane
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t tS = tl + 128u * (uint32_t)t, tO = tl + 256u + 128u * (uint32_t)t;
    uint32_t jobs = 0;                             // key tiles of this stream so far
    uint32_t tiles_before = 0;                     // key tiles of the pieces before
    uint32_t np = 0;                               // pieces so far that see any key
    bool ok = true;
    int32_t* my_meta = a.meta + 12 * (c + 1);
    if (threadIdx.x == 0) my_meta[0] = 0;
    const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
    uint8_t* stage = sm + Sh::kOutOff + 2048 * warp;   // 64 bytes of 32 rows
    int block = -1, token = 0, group = 0, lo = 0, hi = 0;      // of the row, while the row block is the same
    Whole all{0, 0};
    auto stream_wait = [&](int which, uint32_t parity) -> bool {
      return __all_sync(0xFFFFFFFFu, mbar_wait(bar(which), parity & 1u, limit, abort_flag));
    };
    Piece p;
    while (ok && next_piece<kRows>(a, ps, p)) {
      const Item& it = p.it;
      const int row = (kTiles == 2 ? 128 * t : 0) + r;             // row of the item
      const bool live = row < it.rows;
      if (p.block != block) {
        block = p.block;
        const int gr = it.row0 + (live ? row : 0);
        token = a.by_group.of(gr), group = gr - token * a.G;
        const int pos = it.L - it.n + token;
        lo = low_key(a, pos), hi = high_key(a, it.L, pos);
        all = whole_tiles(a, it);
      }
      const int head = p.hk * a.G + group;
      const bool warp_live = (kTiles == 2 ? 128 * t : 0) + 32 * (warp & 3) < it.rows;
      const bool empty = it.tiles == 0;
      const int step = kTiles == 2 ? 1 : 2, j0 = kTiles == 2 ? 0 : t;
      const int mine = empty ? 0 : kTiles == 2 ? (128 * t < it.rows ? p.len : 0) : (p.len + 1 - t) / 2;   // key tiles
      float m = -INFINITY, l = 0.f;
      for (int i = 0; ok && i < mine; ++i, ++jobs) {
        const int j = j0 + step * i, tile = it.tile0 + p.t0 + j;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {              // half a tile: 64 keys, buffer h
          ok = ok && stream_wait(kSFull + 2 * t + h, jobs);
          if (!ok) break;
          if (warp_live) {
            tc_fence_after();
            uint32_t x[64];
            tmem_load(tS + 64u * (uint32_t)h, x);
            // which of the keys the row sees
            const uint2 have = *reinterpret_cast<const uint2*>(mask_s + 4 * ((tiles_before + (uint32_t)j) & 7u) + 2 * h);
            if (!all.has(tile) || (have.x & have.y) != ~0u) {      // (the same for every lane)
              const int k0 = tile * kKeys + 64 * h;
              const uint32_t see0 = have.x & bits_between(lo - k0, hi - k0), see1 = have.y & bits_between(lo - k0 - 32, hi - k0 - 32);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                x[e] = (see0 >> e) & 1u ? x[e] : __float_as_uint(-INFINITY);
                x[32 + e] = (see1 >> e) & 1u ? x[32 + e] : __float_as_uint(-INFINITY);
              }
            }
            float top[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) top[q] = fmaxf(__uint_as_float(x[q]), __uint_as_float(x[8 + q]));
#pragma unroll
            for (int e = 16; e < 64; e += 16)
#pragma unroll
              for (int q = 0; q < 8; ++q) top[q] = fmaxf(fmaxf(top[q], __uint_as_float(x[e + q])), __uint_as_float(x[e + 8 + q]));
#pragma unroll
            for (int q = 0; q < 4; ++q) top[q] = fmaxf(top[q], top[4 + q]);
            const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
            const bool moves = mt > m + kLazy;
            if (__any_sync(0xFFFFFFFFu, moves)) {
              const float f = moves ? ex2(m - mt) : 1.f;
              if (moves) {
                m = mt;
                l *= f;
              }
              if (i > 0 || h > 0) {                // the products of the half tile before have added to O
                ok = h == 0 ? stream_wait(kODone + 2 * t + 1, jobs - 1u) : stream_wait(kODone + 2 * t, jobs);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int cc = 0; cc < D; cc += 32) {
                  uint32_t o[32];
                  tmem_load(tO + (uint32_t)cc, o);
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_store(tO + (uint32_t)cc, o);
                }
              }
            }
            const float mm = m == -INFINITY ? 0.f : m;
            const uint64_t neg = pack2(-mm, -mm);
            uint64_t sum2 = 0;
            uint32_t pw[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float pa, pb;
              unpack2(fma2(pack2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), scale2, neg), pa, pb);
              pa = ex2(pa);
              pb = ex2(pb);
              sum2 = add2(sum2, pack2(pa, pb));
              const __nv_bfloat162 w = __floats2bfloat162_rn(pa, pb);
              pw[e] = *reinterpret_cast<const uint32_t*>(&w);
            }
            tmem_store(tS + 64u * (uint32_t)h, pw);
            float la, lb;
            unpack2(sum2, la, lb);
            l += la + lb;
            tmem_st_wait();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kPFull + 2 * t + h));
        }
      }
      // ---- the item's rows (or its part of them)
      const bool whole = p.t0 == 0 && p.len == p.cost;
      const int slot = p.t0 == 0 ? 2 * c + 1 : 2 * c;
      if (!whole && p.t0 == 0 && threadIdx.x == 0) {               // the item's first part: it owns the sum
        my_meta[1] = it.s, my_meta[2] = it.row0, my_meta[3] = it.rows, my_meta[4] = p.hk;
        my_meta[5] = (int)(((ps.x + (p.cost - p.t0 - p.len)) * C - 1) / line);                // the CTA that holds its last tile
        my_meta[8] = (int32_t)(uint32_t)line, my_meta[9] = (int32_t)(line >> 32);
        my_meta[0] = 1;
      }
      if (ok && mine > 0) ok = stream_wait(kODone + 2 * t + 1, jobs - 1u);
      float m2 = -INFINITY, l2 = 0.f;                              // one row tile: the other stream's
      if constexpr (kTiles == 1) {
        stat_s[128 * t + r] = make_float2(m, l);
        ok = all_well(2, 256, ok);
        const float2 o = stat_s[128 * (t ^ 1) + r];
        m2 = o.x, l2 = o.y;
      }
      if (!ok) break;
      tc_fence_after();
      if (warp_live) {
        // weights of the streams' sums (two where each has had tiles), and the joint statistics
        const bool other = kTiles == 1 && !empty && p.len > 1;
        float f0 = 1.f, f1 = 0.f;                                  // of the only sum, or of stream 0's and 1's
        if (kTiles == 1) {
          const float M = fmaxf(m, m2);
          const float fm = M == -INFINITY ? 1.f : ex2(m - M), fo = M == -INFINITY ? 1.f : ex2(m2 - M);
          l = t == 0 ? l * fm + l2 * fo : l2 * fo + l * fm;
          f0 = t == 0 ? fm : fo;
          f1 = t == 0 ? fo : fm;
          m = M;
        }
        const bool writer = kTiles == 2 || t == 0;
        const float sn = a.sink != nullptr ? a.sink[head] : -INFINITY, sk = sn * kLog2e;
        if (whole) {
          const float top = fmaxf(m, sk);
          float inv;
          if (top == -INFINITY && !(l != l) && !(sn != sn)) {
            inv = 0.f;
            l = sn;                                                // lse (a sink near the lowest fp32 has no base-2 form)
          } else {
            const float g = ex2(m - top), den = l * g + (sk == top ? 1.f : ex2(sk - top));    // (the sink may be infinite)
            inv = g / den;
            l = (sk >= m ? sn : m * kLn2) + logf(den);
          }
          f0 *= inv, f1 *= inv;
          if (a.lse != nullptr && live && writer) a.lse[(int64_t)(it.s + token) * a.H + head] = l;
        } else if (live && writer) {
          reinterpret_cast<float2*>(a.ml)[(int64_t)slot * kRows + row] = make_float2(m, l);
        }
        const bool bad = !empty && bad_s[np & 15u] != 0;
        const int least_hi = bad ? high_key(a, it.L, it.L - it.n + a.by_group.of(it.row0)) : 0;
        const int most_lo = bad ? low_key(a, it.L - it.n + a.by_group.of(it.row0 + it.rows - 1)) : 0;
        constexpr int kCols = kTiles == 2 ? D : D / 2;             // of this warp; one row tile: half each
        constexpr int kW = 32;
        const int c0 = kTiles == 2 ? 0 : t * kCols;
        // where the rows that the lane writes begin, and how many rows the warp has
        const int live_rows = min(32, it.rows - (row - lane));
        const int64_t at = (int64_t)(it.s + token) * a.ldo + (int64_t)head * D;
        int64_t to[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = __shfl_sync(0xFFFFFFFFu, at, 8 * i + (lane >> 2));
        const uint32_t tA = kTiles == 2 ? tO : tl + 256u;          // the only sum, or stream 0's
#pragma unroll 1                                 // (unrolled, its instructions' fetch takes longer than their work)
        for (int cc = 0; cc < kCols; cc += kW) {
          float o[kW];
          {
            uint32_t w[kW];
#pragma unroll
            for (int e = 0; e < kW; ++e) o[e] = 0.f;
            if (!empty) {
              tmem_load(tA + (uint32_t)(c0 + cc), w);
#pragma unroll
              for (int e = 0; e < kW; ++e) o[e] = __uint_as_float(w[e]) * f0;
            }
            if (other) {
              tmem_load(tl + 384u + (uint32_t)(c0 + cc), w);
#pragma unroll
              for (int e = 0; e < kW; ++e) o[e] = fmaf(__uint_as_float(w[e]), f1, o[e]);
            }
          }
          if (bad && live) {
            // values that are no numbers were taken out of the tiles that some row sees in part: the rows that see them
            // get them back, as sums with them give
            for (int j = 0; j < p.len; ++j) {
              const int tile = it.tile0 + p.t0 + j;
              if (all.has(tile)) continue;
              for (int64_t key = max((int64_t)tile * kKeys, (int64_t)lo); key < min((int64_t)(tile + 1) * kKeys, (int64_t)hi); ++key) {
                // (values of 32 keys that every row sees were left in their place)
                if (key / 32 * 32 >= most_lo && key / 32 * 32 + 32 <= least_hi) continue;
                const int blk = a.table[it.b * a.bt_stride + key / a.block_size];
                if (blk < 0 || blk >= a.num_blocks) continue;
                const uint16_t* v = a.v + blk * a.block_stride + key % a.block_size * a.row_stride + p.hk * a.head_stride + c0 + cc;
#pragma unroll
                for (int e = 0; e < kW; ++e)
                  if ((v[e] & 0x7F80u) == 0x7F80u) o[e] += __uint_as_float((uint32_t)v[e] << 16);
              }
            }
          }
          // 64 bytes of each row go through shared memory, so that four lanes write a row's 64 neighbouring bytes (a row
          // per lane made the writes of 256 rows take 5 us): piece q of row r at q ^ (r / 2 % 4), free of conflicts
          auto put = [&](const uint4 (&v)[4], auto place) {
#pragma unroll
            for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(stage + 64 * lane + 16 * (q ^ (lane >> 1 & 3))) = v[q];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rr = 8 * i + (lane >> 2), q = lane & 3;
              const uint4 w = *reinterpret_cast<const uint4*>(stage + 64 * rr + 16 * (q ^ (rr >> 1 & 3)));
              if (rr < live_rows) *reinterpret_cast<uint4*>(place(i, rr) + 16 * q) = w;
            }
            __syncwarp();
          };
          uint4 v[4];
          if (whole) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(o[8 * q + 2 * i], o[8 * q + 2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
              }
              v[q] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            put(v, [&](int i, int) { return reinterpret_cast<uint8_t*>(a.out + to[i] + c0 + cc); });
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                v[q] = make_uint4(__float_as_uint(o[e + 4 * q]), __float_as_uint(o[e + 4 * q + 1]),
                                  __float_as_uint(o[e + 4 * q + 2]), __float_as_uint(o[e + 4 * q + 3]));
              put(v, [&](int, int rr) {
                return reinterpret_cast<uint8_t*>(a.part + ((int64_t)slot * kRows + row - lane + rr) * D + c0 + cc + e);
              });
            }
          }
        }
        tc_fence_before();
      }
      if constexpr (kTiles == 1) ok = all_well(2, 256, ok);       // both streams' sums have been read
      if (!empty) {
        tiles_before += (uint32_t)p.len;
        ++np;
      }
    }
    if (!ok && lane == 0) {
      raise_error(DSA_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
  } else if (warp < 12) {
    // ================================ keys and values ================================
    // Lane l of warp w resolves row 32 w + l of each tile; lanes whose row begins a copy issue it (both halves of 128
    // dims by lanes of their own).
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    constexpr int kHalves = D / 64;
    const int w32 = 32 * (warp & 3);
    const int box = a.box, units = (box == 1 ? 8 : box >= 32 ? (w32 % box == 0 ? 1 : 0) : 32 / box) * kHalves;
    const int unit_row = lane / kHalves * (box == 1 ? 4 : box >= 32 ? 32 : box);   // the lane's copy: its first row in the warp
    const uint32_t unit_dst = (uint32_t)(lane % kHalves) * 16384u + (uint32_t)(w32 + unit_row) * 128u;
    const int unit_x = 64 * (lane % kHalves);
    const uint32_t bytes = (uint32_t)(box == 1 ? 512 : 128 * box) * (uint32_t)units;
    uint32_t loads = 0, tiles = 0, np = 0, looks = 0;
    bool ok = true;
    Piece p;
    while (ok && next_piece<kRows>(a, ps, p)) {
      const Item& it = p.it;
      if (it.tiles == 0) continue;
      const int first = it.tile0 + p.t0;
      const Whole all = whole_tiles(a, it);
      const int32_t* table = a.table + (int64_t)it.b * a.bt_stride;
      // the lane's key, its page and place in it, and the page's block, one tile ahead (-1: no copy brings it)
      int64_t key = (int64_t)first * kKeys + w32 + lane;
      uint32_t page = (uint32_t)a.by_block.of((int)min(key, (int64_t)INT32_MAX)), off = (uint32_t)key - page * (uint32_t)a.block_size;
      const uint32_t page_step = kKeys / (uint32_t)a.block_size, off_step = kKeys % (uint32_t)a.block_size;
      auto block_of = [&](int j) {
        const int64_t from = key & -(int64_t)box;
        return j < p.len && from + box > it.lo && from < it.hi ? table[page] : -1;
      };
      int blk = block_of(0);
      int y = a.no_row, y1 = a.no_row;             // the lane's row in this tile and the one before it
      const int x = p.hk * a.head_cols + unit_x, y0 = p.hk * a.head_rows;
      if (warp == 8 && lane == 0) bad_s[np & 15u] = 0;
      auto rows_of = [&](int j) {
        const bool seen = key >= it.lo && key < it.hi;
        const bool there = blk >= 0 && blk < a.num_blocks;
        if (seen && !there) raise_error(DSA_DEVERR_INDEX);
        y1 = y;
        y = there ? blk * a.block_rows + y0 + (int)off : a.no_row;
        const uint32_t word = __ballot_sync(0xFFFFFFFFu, there);
        if (lane == 0) mask_s[4 * ((tiles + (uint32_t)j) & 7u) + (uint32_t)(warp & 3)] = word;
        key += kKeys;
        page += page_step, off += off_step;
        if (off >= (uint32_t)a.block_size) off -= (uint32_t)a.block_size, ++page;
        blk = block_of(j + 1);
      };
      // copies announce themselves to the products, or, for values that are looked through, to those who look
      auto bring = [&](const CUtensorMap* tm, int row, bool look) {
        const int st = (int)(loads % kStages);
        ok = mbar_wait(bar(kEmpty + st), (loads / kStages & 1u) ^ 1u, limit, abort_flag);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) return;
        const uint32_t to = bar(look ? kLook + (int)(looks & 7u) : kFull + st);
        if (look) ++looks;
        if (lane == 0) mbar_arrive_expect_tx(to, bytes);
        const uint32_t dst = sm32 + Sh::kStageOff + (uint32_t)st * Sh::kTile + unit_dst;
        if (box == 1) {
          int rows[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) rows[i] = __shfl_sync(0xFFFFFFFFu, row, (unit_row + i) & 31);
          if (lane < units) gather4(dst, tm, to, x, rows);
        } else {
          const int at = __shfl_sync(0xFFFFFFFFu, row, unit_row & 31);
          if (lane < units) tma_load_2d(dst, tm, to, x, at);
        }
        __syncwarp();
        ++loads;
      };
      if constexpr (kTiles == 2) {
        for (int j = 0; ok && j < p.len; ++j) {
          rows_of(j);
          bring(&tmk, y, false);
          if (ok) bring(&tmv, y, !all.has(first + j));
        }
      } else {                                     // keys two tiles ahead of the values
        for (int j = 0; ok && j < p.len; ++j) {
          if (j >= 2) bring(&tmv, y1, !all.has(first + j - 2));
          if (!ok) break;
          rows_of(j);
          bring(&tmk, y, false);
        }
        if (ok && p.len >= 2) bring(&tmv, y1, !all.has(first + p.len - 2));
        if (ok) bring(&tmv, y, !all.has(first + p.len - 1));
      }
      tiles += (uint32_t)p.len;
      ++np;
    }
    if (!ok && lane == 0) {
      raise_error(DSA_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
    // every copy issued has landed before the CTA may leave
    // (where others have given up, a stage may never fill; after one such wait all have landed)
    for (uint32_t i = loads > (uint32_t)kStages ? loads - kStages : 0; i < loads; ++i)
      if (!mbar_wait(bar(kFull + (int)(i % kStages)), i / kStages & 1u, kCleanupWaitNs, nullptr)) break;
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp < 14) {
      // ================================ products ================================
      // A warp per stream; its control flow is the same for all lanes (and the compiler can tell: what it depends on is
      // broadcast), so that the operands of a product are uniform and cost an addition each.  With one thread branching
      // off on its own, issuing the products of a tile took 3.4 times as long, and longer than the products.
      constexpr uint32_t kIdescS = idesc_bf16(128, 64), kIdescO = idesc_bf16(128, D) | (1u << 16);   // V: dims contiguous
      const uint32_t t = (uint32_t)__shfl_sync(0xFFFFFFFFu, warp - 12, 0), tq = kTiles == 2 ? t : 0;
      const uint32_t tb = __shfl_sync(0xFFFFFFFFu, tmem, 0), smb = __shfl_sync(0xFFFFFFFFu, sm32, 0);
      const uint32_t bs = smb + Sh::kBarOff;
      const bool mine = elect_one();
      // Every stage is released by both streams, also by one that has no use for it: a barrier's phases are told apart by
      // their parity, so whoever waits on one has to pass all of them.
      uint32_t base = 0, pieces = 0, jobs = 0, next = 0;
      bool ok = true;
      auto wait = [&](uint32_t which, uint32_t parity) -> bool {
        return (bool)__all_sync(0xFFFFFFFFu, mbar_wait(bs + 8u * which, parity, limit, abort_flag));
      };
      Piece p;
      while (ok && next_piece<kRows>(a, ps, p)) {
        const uint32_t len = __shfl_sync(0xFFFFFFFFu, p.len, 0);
        const bool two = __shfl_sync(0xFFFFFFFFu, p.it.rows, 0) > 128, empty = __shfl_sync(0xFFFFFFFFu, p.it.tiles, 0) == 0;
        if (empty) continue;
        const uint32_t n = kTiles == 2 ? (t == 0 || two ? len : 0) : (len + 1 - t) / 2;   // the stream's jobs
        auto take = [&](uint32_t ld) {             // waits for a load, releasing the other stream's before it
          for (; next < ld; ++next) {
            if (!wait(kFull + next % kStages, next / kStages & 1u)) return false;
            if (mine) mbar_arrive(bs + 8u * (kEmpty + next % kStages));
          }
          return wait(kFull + ld % kStages, ld / kStages & 1u);
        };
        // job 2 i + h: keys 64 h .. of the stream's key tile i, buffer h.  Loads come in the order K0 V0 K1 V1 .. or
        // K0 K1 V0 K2 V1 ..
        auto tile = [&](uint32_t i) { return kTiles == 2 ? i : 2 * i + t; };
        auto scores = [&](uint32_t i, uint32_t h) -> bool {
          const uint32_t j = tile(i), ld = base + (kTiles == 2 ? 2 * j : j < 2 ? j : 2 * j - 1), s = ld % kStages;
          if (h == 0) {
            if (!take(ld)) return false;
            next = ld + 1;
            tc_fence_after();
          }
          const uint32_t qa = desc_low(smb + tq * Sh::kTile, 0), ka = desc_low(smb + Sh::kStageOff + s * Sh::kTile + 8192u * h, 0);
          if (mine) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((uint32_t)(kk >> 2) * 16384u + (uint32_t)(kk & 3) * 32u) >> 4;
              if (kk == 0) mma_ss<false>(tb + 128u * t + 64u * h, qa, ka, kIdescS);
              else mma_ss<true>(tb + 128u * t + 64u * h, qa + off, ka + off, kIdescS);
            }
            mma_commit(bs + 8u * (kSFull + 2 * t + h));
            if (h == 1) {
              mma_commit(bs + 8u * (kEmpty + s));
              if (i == n - 1) mma_commit(bs + 8u * (kQFree + tq));
            }
          }
          __syncwarp();
          return true;
        };
        if (n > 0 || kTiles == 1) {
          ok = wait(kQFull + tq, pieces & 1u);
          ++pieces;
          if (ok && n > 0) ok = scores(0, 0) && scores(0, 1);
          else if (ok && mine) mbar_arrive(bs + 8u * kQFree);
        }
        for (uint32_t i = 0; ok && i < n; ++i, ++jobs) {
          const uint32_t j = tile(i);
          const uint32_t ld = base + (kTiles == 2 ? 2 * j + 1 : min(2 * j + 2, 2 * len - 1)), s = ld % kStages;
          ok = take(ld);
          next = ld + 1;
          const uint32_t va = desc_low(smb + Sh::kStageOff + s * Sh::kTile, 16384u);
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h) {
            ok = ok && wait(kPFull + 2 * t + h, jobs & 1u);
            if (!ok) break;
            tc_fence_after();
            if (mine) {
#pragma unroll
              for (uint32_t kk = 0; kk < 4; ++kk)
                mma_ts(tb + 256u + 128u * t, tb + 128u * t + 64u * h + 8u * kk, va + (4 * h + kk) * (2048u >> 4), kIdescO,
                       h == 0 && kk == 0 ? (i > 0 ? 1u : 0u) : 1u);
              mma_commit(bs + 8u * (kODone + 2 * t + h));
              if (h == 1) mma_commit(bs + 8u * (kEmpty + s));
            }
            __syncwarp();
            if (i + 1 < n) ok = scores(i + 1, h);
          }
        }
        base += 2u * len;
        if (ok && next < base) {                   // what the other stream has left
          ok = take(base - 1);
          if (ok && mine) mbar_arrive(bs + 8u * (kEmpty + (base - 1) % kStages));
          next = base;
        }
      }
      if (!ok && lane == 0) {
        raise_error(DSA_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      if (mine) mma_commit(bs + 8u * (kDrain + t));      // everything issued has completed
      mbar_wait(bs + 8u * (kDrain + t), 0u, kCleanupWaitNs, nullptr);
    } else {
      // ================================ queries, and a look at values ================================
      // Where some row sees a tile in part, its values that are no numbers are taken out (a zero weight would not silence
      // them); the rows that do see them get them back with the sums.  Keys outside the item's
      // range need no more: finite values under a zero weight are nothing.
      uint32_t base = 0, looked = 0, np = 0, loads0 = 0, loads1 = 0;
      const int lt = (int)threadIdx.x - 14 * 32;
      int block = -1, least_hi = 0, most_lo = 0;
      Whole all{0, 0};
      bool ok = true;
      Piece p;
      while (ok && next_piece<kRows>(a, ps, p)) {
        const Item& it = p.it;
        if (it.tiles == 0) continue;
        for (int t = 0; ok && t < (kTiles == 2 && it.rows > 128 ? 2 : 1); ++t) {
          constexpr int kPer = D / 8, kStep = 64 / kPer;
          ok = mbar_wait(bar(kQFree + t), ((t == 0 ? loads0 : loads1) & 1u) ^ 1u, limit, abort_flag);
          ok = all_well(1, 64, ok);                // both warps have seen it: the copy may bring its next phase about
          if (!ok) break;
          if (t == 0) ++loads0;
          else ++loads1;
          if (a.q_boxes) {
            if (lt == 0) {
              mbar_arrive_expect_tx(bar(kQFull + t), Sh::kTile);
              const int token = it.s + a.by_group.of(it.row0 + 128 * t);
              for (int h = 0; h < D / 64; ++h)
                tma_load_3d(sm32 + (uint32_t)t * Sh::kTile + 16384u * (uint32_t)h, &tmq, bar(kQFull + t), 64 * h, p.hk * a.G, token);
            }
            continue;
          }
          // row tiles that are no boxes: a piece of 16 bytes per thread and pass
          const int pc = lt % kPer, r0 = lt / kPer;
          const int first = it.row0 + 128 * t + r0, left = it.rows - 128 * t - r0;   // rows from the thread's first on
          const int token = a.by_group.of(first);
          uint32_t g = (uint32_t)(first - token * a.G);
          // from row to row: kStep heads on, which is `more` tokens and `on` heads, or one token more and G heads less
          const int more = a.by_group.of(kStep);
          const uint32_t on = (uint32_t)(kStep - more * a.G);
          const uint16_t* src = a.q + (int64_t)(it.s + token) * a.ldq + (int64_t)(p.hk * a.G + (int)g) * D + pc * 8;
          const int64_t hop = more * a.ldq + (int64_t)on * D, wrap = a.ldq - (int64_t)a.G * D;
          const uint32_t dst = sm32 + (uint32_t)t * Sh::kTile + (uint32_t)(pc >> 3) * 16384u + (uint32_t)r0 * 128u;
#pragma unroll 4
          for (int i = 0; i < 128 / kStep; ++i) {
            const bool live = i * kStep < left;
            copy16(dst + (uint32_t)(i * kStep) * 128u + (uint32_t)(((pc & 7) ^ ((r0 + i * kStep) & 7)) << 4), live ? src : a.q, live);
            src += hop, g += on;
            if (g >= (uint32_t)a.G) g -= (uint32_t)a.G, src += wrap;
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        }
        if (!a.q_boxes && !ok) asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (!a.q_boxes && ok) {
          if (kTiles == 2 && it.rows > 128) {      // the first tile's may be used before the second's are there
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            proxy_fence();
            mbar_arrive(bar(kQFull));
          }
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          proxy_fence();
          mbar_arrive(bar(kQFull + (kTiles == 2 && it.rows > 128 ? 1 : 0)));
        }
        if (p.block != block) {
          block = p.block;
          all = whole_tiles(a, it);
          least_hi = high_key(a, it.L, it.L - it.n + a.by_group.of(it.row0));
          most_lo = low_key(a, it.L - it.n + a.by_group.of(it.row0 + it.rows - 1));
        }
        for (int j = 0; ok && j < p.len; ++j) {
          const int tile = it.tile0 + p.t0 + j;
          if (all.has(tile)) continue;
          const uint32_t ld = base + (uint32_t)(kTiles == 2 ? 2 * j + 1 : min(2 * j + 2, 2 * p.len - 1)), st = ld % kStages;
          ok = mbar_wait(bar(kLook + (int)(looked & 7u)), looked >> 3 & 1u, limit, abort_flag);
          ok = __all_sync(0xFFFFFFFFu, ok);
          ++looked;
          if (ok) {
            // Thread: 16-byte column lt % 8 of every eighth row, half by half.  A half word is no number where its
            // exponent's bits are all set: then adding one in the lowest of them carries into the sign's place.
            uint8_t* at = sm + Sh::kStageOff + st * Sh::kTile + (lt >> 3) * 128 + (lt & 7) * 16;
            const int64_t k0 = (int64_t)tile * kKeys + (lt >> 3);
            bool found = false;
#pragma unroll 1
            for (int i0 = 0; i0 < 16; i0 += 4) {   // 32 keys; those that every row sees need no look
              const int64_t first = (int64_t)tile * kKeys + 8 * i0;
              if (first >= most_lo && first + 32 <= least_hi) continue;
              uint4 w[4 * (D / 64)];
#pragma unroll
              for (int i = 0; i < 4 * (D / 64); ++i) w[i] = *reinterpret_cast<uint4*>(at + 1024 * (i0 + (i & 3) + 16 * (i >> 2)));
              uint32_t any = 0;
#pragma unroll
              for (int i = 0; i < 4 * (D / 64); ++i)
                any |= ((w[i].x & 0x7F807F80u) + 0x00800080u) | ((w[i].y & 0x7F807F80u) + 0x00800080u) |
                       ((w[i].z & 0x7F807F80u) + 0x00800080u) | ((w[i].w & 0x7F807F80u) + 0x00800080u);
              if ((any & 0x80008000u) == 0) continue;
#pragma unroll 1
              for (int i = 0; i < 4 * (D / 64); ++i) {
                const int64_t key = k0 + 8 * (i0 + (i & 3));
                uint32_t* here = reinterpret_cast<uint32_t*>(at + 1024 * (i0 + (i & 3) + 16 * (i >> 2)));
                for (int e = 0; e < 4; ++e) {
                  const uint32_t v = here[e];
                  uint32_t u = v;
                  if ((u & 0x7F80u) == 0x7F80u) u &= 0xFFFF0000u;
                  if ((u & 0x7F800000u) == 0x7F800000u) u &= 0x0000FFFFu;
                  if (u != v) {
                    here[e] = u;
                    found |= key >= it.lo && key < it.hi;
                  }
                }
              }
            }
            if (found) bad_s[np & 15u] = 1;
            proxy_fence();
          }
          ok = all_well(1, 64, ok);                // both halves are done
          if (ok && lt == 0) mbar_arrive_n(bar(kFull + (int)st), 4);
        }
        base += 2u * (uint32_t)p.len;
        ++np;
      }
      if (!ok && lane == 0) {
        raise_error(DSA_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      if (a.q_boxes && loads0 > 0) mbar_wait(bar(kQFull), (loads0 - 1) & 1u, kCleanupWaitNs, nullptr);
      if (a.q_boxes && loads1 > 0) mbar_wait(bar(kQFull + 1), (loads1 - 1) & 1u, kCleanupWaitNs, nullptr);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

// Adds the parts of the items that slice ends have cut, in the order of their keys:
//   M = max(m_p, sink), out = sum_p 2^(m_p - M) O_p / (sum_p 2^(m_p - M) l_p + 2^(sink - M)).
// Block c: the item whose first part is CTA c's (at most one); a warp per row.
template <int D, int kRows>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ AttnArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int c = (int)blockIdx.x, lane = (int)threadIdx.x & 31;
  const int4* meta = reinterpret_cast<const int4*>(a.meta) + 3 * (c + 1);
  const int4 m0 = meta[0], m1 = meta[1], m2 = meta[2];       // split, first token's row, first row, rows; key head, last CTA; line
  if (m0.x == 0) return;
  const int hk = m1.x, parts = m1.y - c + 1;
  const int64_t line = (int64_t)(uint32_t)m2.x | (int64_t)m2.y << 32, C = gridDim.x;
  // Part i is in the owner's second slot or CTA c + i's first; a CTA without any of the line (more CTAs than tiles) has none.
  const auto slot = [](int i) { return i == 0 ? 1 : 2 * i; };        // from the owner's first
  const bool dense = line >= C;
  const auto is_part = [&](int i) {
    return i < parts && (i == 0 || dense || line * (c + i) / C < line * (c + i + 1) / C);
  };
  constexpr int kE = D / 32, kAhead = 4;
  for (int row = (int)(blockIdx.y * 8 + (threadIdx.x >> 5)); row < m0.w; row += (int)gridDim.y * 8) {
    const int token = a.by_group.of(m0.z + row), head = hk * a.G + (m0.z + row) - token * a.G;
    const float sn = a.sink != nullptr ? a.sink[head] : -INFINITY, sk = sn * kLog2e;
    const float2* ml = reinterpret_cast<const float2*>(a.ml) + (int64_t)2 * c * kRows + row;
    const float* sums = a.part + ((int64_t)2 * c * kRows + row) * D + lane * kE;
    float acc[kE], M = sk, den = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] = 0.f;
    // 32 parts at a time, their statistics a lane each; the sums so far move with the maximum
    for (int i0 = 0; i0 < parts; i0 += 32) {
      const bool there = is_part(i0 + lane);
      const uint32_t have = __ballot_sync(0xFFFFFFFFu, there);
      const float2 s = there ? ml[slot(i0 + lane) * kRows] : make_float2(-INFINITY, 0.f);
      const int n = min(32, parts - i0);
      float w = 1.f;
      for (int k0 = 0; k0 < n; k0 += kAhead) {
        float o[kAhead][kE];                       // on their way while the weights are found
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
#pragma unroll
          for (int e = 0; e < kE; ++e) o[k][e] = 0.f;
          if (have >> (k0 + k) & 1u) {             // (k0 + k <= 31)
            const float* from = sums + slot(i0 + k0 + k) * (kRows * D);
            if constexpr (kE == 4) {
              const float4 v = *reinterpret_cast<const float4*>(from);
              o[k][0] = v.x, o[k][1] = v.y, o[k][2] = v.z, o[k][3] = v.w;
            } else {
              const float2 v = *reinterpret_cast<const float2*>(from);
              o[k][0] = v.x, o[k][1] = v.y;
            }
          }
        }
        if (k0 == 0) {
          float top = s.x;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
          top = fmaxf(top, M);
          const float old = top == M ? 1.f : ex2(M - top);
          M = top;
          w = !there ? 0.f : M == -INFINITY ? 1.f : ex2(s.x - M);
          float part = there ? s.y * w : 0.f;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, d);
          den = den * old + part;
#pragma unroll
          for (int e = 0; e < kE; ++e) acc[e] *= old;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {         // (lanes past the parts hold no weight)
          const float f = __shfl_sync(0xFFFFFFFFu, w, k0 + k);
#pragma unroll
          for (int e = 0; e < kE; ++e) acc[e] = fmaf(o[k][e], f, acc[e]);
        }
      }
    }
    const bool none = M == -INFINITY && !(den != den);
    den += M == -INFINITY ? 0.f : sk == M ? 1.f : ex2(sk - M);
    const float inv = none ? 0.f : 1.f / den;
    uint16_t* dst = a.out + (int64_t)(m0.y + token) * a.ldo + (int64_t)head * D + lane * kE;
#pragma unroll
    for (int e = 0; e < kE; e += 2)
      *reinterpret_cast<__nv_bfloat162*>(dst + e) = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
    if (a.lse != nullptr && lane == 0) a.lse[(int64_t)(m0.y + token) * a.H + head] = none ? sn : (sk >= M ? sn : M * kLn2) + logf(den);
  }
}

Divisor divisor(int d) {
  int s = 0;
  while (((int64_t)1 << s) < d) ++s;
  return {(uint32_t)((((uint64_t)1 << (31 + s)) + (uint64_t)d - 1) / (uint64_t)d), 31 + s};
}

struct Layout {
  int tiles, rows, ctas;
  int64_t blocks;
  size_t meta, ml, part, prefix, first, seq, total;
};

// Two row tiles where a sequence brings more than one on average: each key tile then feeds twice the products.  (8192-token
// prompt 734 us, with one 908; one token over 4096 keys 15.6 us with two, 12.8 with one.)
int row_tiles(int64_t T, int B, int H, int Hkv) { return T * (H / Hkv) > 128 * (int64_t)B ? 2 : 1; }

Layout layout(int tiles, int64_t T, int B, int H, int Hkv, int D, int num_sms) {
  Layout y{};
  const int64_t G = H / Hkv;
  y.tiles = tiles;
  y.rows = 128 * y.tiles;
  y.ctas = num_sms;
  const int64_t blocks = T * G / y.rows + (B < T ? B : T);        // at most so many row blocks
  y.blocks = blocks;
  const auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  y.meta = 0;
  y.ml = up(48 * (size_t)(y.ctas + 1));
  y.part = y.ml + up((size_t)2 * y.ctas * y.rows * 8);
  y.prefix = y.part + up((size_t)2 * y.ctas * y.rows * D * 4);
  y.first = y.prefix + up(8 * (size_t)(blocks + 1));
  y.seq = y.first + up(4 * (size_t)B);
  y.total = y.seq + up(4 * (size_t)blocks);
  return y;
}

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// bf16 tensors of two or three dimensions in boxes of 64 elements (128-byte swizzle).  What lies outside reads as zeros.
bool make_map(CUtensorMap* m, const void* base, int dims, const cuuint64_t* size, const cuuint64_t* strides, const cuuint32_t* box) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)dims, const_cast<void*>(base), size, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
  CUtensorMap q, k, v;
};

template <int D, int kTiles>
cudaError_t launch_shape(const AttnArgs& a, const Maps& m, int ctas, cudaStream_t stream) {
  using Sh = Shape<D, kTiles>;
  auto kernel = paged_attn_kernel<D, kTiles>;
  static std::atomic<unsigned long long> ready{0};               // devices on which the kernel is set up
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1u)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Sh::kSmem);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    // the warps' shares, 2 x 168 + 2 x 88 registers a thread, are those of the launch
    if (fa.numRegs * kThreads < 128 * (2 * 168 + 2 * 88)) return cudaErrorInvalidConfiguration;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  if (a.planned) {
    e = launch_pdl(plan_kernel<Sh::kRows>, dim3(1), 1024u, 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(kernel, dim3((unsigned)ctas), (unsigned)kThreads, Sh::kSmem, stream, m.q, m.k, m.v, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(combine_kernel<D, Sh::kRows>, dim3((unsigned)ctas, Sh::kRows / 8), 256u, 0, stream, a);
}

}  // namespace

bool paged_attn_cache_fits(const dsa_kv_cache& kv, int Hkv) {
  if (kv.block_stride % kv.row_stride != 0) return false;
  if (Hkv > 1 && kv.head_stride > kv.row_stride && kv.head_stride % kv.row_stride != 0) return false;
  if (Hkv > 1 && kv.head_stride < kv.row_stride && (int64_t)Hkv * kv.head_stride > INT32_MAX) return false;
  const int64_t head_rows = Hkv > 1 && kv.head_stride >= kv.row_stride ? kv.head_stride / kv.row_stride : 0;
  const int64_t block_rows = kv.block_stride / kv.row_stride;
  return block_rows <= INT32_MAX / kv.num_blocks && head_rows <= INT32_MAX / Hkv &&
         kv.num_blocks * block_rows + Hkv * head_rows + kv.block_size <= INT32_MAX;
}

size_t paged_attn_ws_bytes(int64_t T, int B, int H, int Hkv, int D, int num_sms) {
  return layout(row_tiles(T, B, H, Hkv), T, B, H, Hkv, D, num_sms).total;
}

// One row tile serves any call, with half the room for parts.  So the size of one step is enough for every smaller one (in
// T and B), whichever takes two: at the same number of tiles the size only grows with T and B, and where the smaller one
// alone takes one tile, its plan's 12 bytes for each of at most 2 B row blocks are less than the parts save.
size_t paged_attn_least_ws_bytes(int64_t T, int B, int H, int Hkv, int D, int num_sms) {
  const size_t one = layout(1, T, B, H, Hkv, D, num_sms).total, own = paged_attn_ws_bytes(T, B, H, Hkv, D, num_sms);
  return one < own ? one : own;
}

cudaError_t launch_paged_attn(const uint16_t* q, int64_t ldq, int64_t T, int H, int Hkv, int D, const int32_t* start,
                              const int32_t* lens, int B, const int32_t* table, int64_t bt_stride, const dsa_kv_cache& kv,
                              float scale, bool causal, int window, const float* sink, uint16_t* out, int64_t ldo, float* lse,
                              void* ws, size_t ws_bytes, int num_sms, cudaStream_t stream) {
  Layout y = layout(row_tiles(T, B, H, Hkv), T, B, H, Hkv, D, num_sms);
  if (ws_bytes < y.total) y = layout(1, T, B, H, Hkv, D, num_sms);
  uint8_t* w = static_cast<uint8_t*>(ws);
  AttnArgs a{};
  a.q = q, a.ldq = ldq, a.start = start, a.lens = lens, a.table = table, a.bt_stride = bt_stride;
  a.v = static_cast<const uint16_t*>(kv.v);
  a.num_blocks = kv.num_blocks, a.block_stride = kv.block_stride, a.row_stride = kv.row_stride, a.head_stride = kv.head_stride;
  a.block_size = kv.block_size;
  a.cap = bt_stride > INT32_MAX / kv.block_size ? INT32_MAX : bt_stride * kv.block_size;
  a.T = T, a.B = B, a.H = H, a.Hkv = Hkv, a.G = H / Hkv;
  a.causal = causal, a.window = window;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.sink = sink, a.out = out, a.ldo = ldo, a.lse = lse;
  a.meta = reinterpret_cast<int32_t*>(w + y.meta);
  a.ml = reinterpret_cast<float*>(w + y.ml);
  a.part = reinterpret_cast<float*>(w + y.part);
  a.prefix = reinterpret_cast<int64_t*>(w + y.prefix);
  a.first = reinterpret_cast<int32_t*>(w + y.first);
  a.seq = reinterpret_cast<int32_t*>(w + y.seq);
  // a CTA plans by itself what fits its shared memory and 32-bit sums
  a.planned = y.blocks > kPlanMax || B > kPlanMax || a.cap > 1 << 29;
  a.limit = (int)y.blocks;
  // the pool as one tensor of rows row_stride apart (paged_attn_cache_fits)
  const bool in_row = Hkv == 1 || kv.head_stride < kv.row_stride;
  a.block_rows = (int)(kv.block_stride / kv.row_stride);
  a.head_cols = in_row && Hkv > 1 ? (int)kv.head_stride : 0;
  a.head_rows = in_row ? 0 : (int)(kv.head_stride / kv.row_stride);
  a.no_row = (int)((kv.num_blocks - 1) * a.block_rows + (int64_t)(Hkv - 1) * a.head_rows + kv.block_size);
  a.box = 1;
  if (kv.block_size % 8 == 0)
    for (a.box = 8; a.box < kKeys && kv.block_size % (2 * a.box) == 0;) a.box *= 2;
  a.q_boxes = 128 % a.G == 0;
  a.by_group = divisor(a.G);
  a.by_block = divisor(kv.block_size);
  Maps m{};
  const cuuint64_t size[2] = {(cuuint64_t)((Hkv - 1) * (int64_t)a.head_cols + D), (cuuint64_t)a.no_row};
  const cuuint64_t stride[1] = {(cuuint64_t)kv.row_stride * 2};
  const cuuint32_t box[2] = {64u, (cuuint32_t)a.box};
  if (!make_map(&m.k, kv.k, 2, size, stride, box) || !make_map(&m.v, kv.v, 2, size, stride, box)) return cudaErrorInvalidValue;
  if (a.q_boxes) {
    const cuuint64_t qsize[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t qstride[2] = {(cuuint64_t)D * 2, (cuuint64_t)ldq * 2};
    const cuuint32_t qbox[3] = {64u, (cuuint32_t)a.G, (cuuint32_t)(128 / a.G)};
    if (!make_map(&m.q, q, 3, qsize, qstride, qbox)) return cudaErrorInvalidValue;
  }
  if (D == 128) return y.tiles == 2 ? launch_shape<128, 2>(a, m, y.ctas, stream) : launch_shape<128, 1>(a, m, y.ctas, stream);
  return y.tiles == 2 ? launch_shape<64, 2>(a, m, y.ctas, stream) : launch_shape<64, 1>(a, m, y.ctas, stream);
}

DSA_DEFINE_TU_ERROR_ACCESSORS(paged_attn)

}  // namespace dsa
