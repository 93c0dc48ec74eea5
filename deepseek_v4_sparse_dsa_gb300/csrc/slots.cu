// Block tables, slot mapping and positions of a step, from request lengths (sm_103a).
//
// Request b holds cached[b] tokens in ceil(cached[b] / bs) pages and brings new[b] more.  Its
// new pages come from the free list in request order, and every new token gets its position
// and its pool row: the two running sums (new tokens, new pages) over the requests decide
// everything.  The data are a few bytes per request and token, so what bounds a step is
// latency: one launch, and no CTA waits for another.  A CTA owns 1024 tokens of the step and
// runs the running sums over all requests itself (8 bytes per request, from L2), keeping the
// requests that have a token in its tile; a token then finds its request by a running
// maximum of head positions.  The token that opens a page writes the page's table entry.
// Measured: 64 requests with a token each 2.9 us, 1000 requests with 8192 tokens 3.9 us, 32 prompts with
// 262144 tokens 4.3 us; every further 1024 requests cost a step of about 1.2 us.
#include "common.cuh"
#include "launch.h"

namespace dsa {
namespace {

constexpr int kSlotThreads = 256;
constexpr int kSlotPer = 4;                              // requests (and tokens) per thread and step
constexpr int kSlotTile = kSlotThreads * kSlotPer;

struct SlotArgs {
  const int32_t* cached;
  const int32_t* fresh;         // new tokens per request
  int B;
  int bs;
  const int32_t* free_blocks;
  int n_free;
  int64_t num_blocks;
  int32_t* table;
  int64_t bt_stride;
  int64_t max_tokens;
  int32_t* context;
  int32_t* start;               // [B + 1]
  int64_t* slot;
  int32_t* pos;
  int32_t* used;
  uint32_t mul, shift;          // division by bs (div_page)
};

__device__ __forceinline__ int32_t clamp_i32(int64_t v) { return v > INT32_MAX ? INT32_MAX : (int32_t)v; }

// Division of 0 <= n < 2^31 by the page size as a product and a shift (division by an invariant integer,
// Granlund and Montgomery): with 2^(s-1) < bs <= 2^s and mul = ceil(2^(31 + s) / bs) <= 2^32 - 1 for
// bs > 1, n mul / 2^(31 + s) exceeds n / bs by less than n / 2^31 < 1 / bs, so its floor is n / bs.
__device__ __forceinline__ int div_page(const SlotArgs& a, int n) {
  return a.bs == 1 ? n : (int)(((uint64_t)(uint32_t)n * a.mul) >> a.shift);
}

// Pages that hold n tokens.
__device__ __forceinline__ int pages(const SlotArgs& a, int n) { return n > 0 ? div_page(a, n - 1) + 1 : 0; }

__device__ __forceinline__ int64_t warp_incl_sum(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

__global__ void __launch_bounds__(kSlotThreads) assign_slots_kernel(const SlotArgs a) {
  constexpr int kWarps = kSlotThreads / 32;
  __shared__ int64_t s_tok[kWarps], s_pg[kWarps];
  __shared__ int s_max[kWarps];
  __shared__ int s_head[kSlotTile];                      // head position of each token's request in the tile
  __shared__ int s_b[kSlotTile], s_old[kSlotTile];       // of the request whose tokens start at this position:
  __shared__ int64_t s_first[kSlotTile];                 //   its first free-list entry
  __shared__ int64_t s_start[kSlotTile];                 //   its first token
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * kSlotTile;
  const int64_t t1 = t0 + kSlotTile < a.max_tokens ? t0 + kSlotTile : a.max_tokens;
  grid_dependency_wait();
#pragma unroll
  for (int i = 0; i < kSlotPer; ++i) s_head[i * kSlotThreads + tid] = -1;
  bool bad = false;
  int64_t tok = 0, pg = 0;                               // running sums before this step's requests
  const int steps = (a.B + kSlotTile - 1) / kSlotTile;
  // The next step's lengths, in flight.  Plain loads: the kernel may be resident before they are written, so the
  // read-only path is not for them.
  int32_t n_next[kSlotPer], old_next[kSlotPer];
  auto fetch = [&](int c) {
#pragma unroll
    for (int i = 0; i < kSlotPer; ++i) {
      const int b = c * kSlotTile + tid * kSlotPer + i;
      n_next[i] = b < a.B ? a.fresh[b] : 0;
      old_next[i] = b < a.B ? a.cached[b] : 0;
    }
  };
  fetch(0);
  for (int c = 0; c < steps; ++c) {
    int32_t n[kSlotPer], old[kSlotPer], need[kSlotPer];
    int64_t ts = 0, ps = 0;
#pragma unroll
    for (int i = 0; i < kSlotPer; ++i) {
      n[i] = n_next[i];
      old[i] = old_next[i];
    }
    if (c + 1 < steps) fetch(c + 1);
#pragma unroll
    for (int i = 0; i < kSlotPer; ++i) {
      const int b = c * kSlotTile + tid * kSlotPer + i;
      need[i] = 0;
      if (b < a.B) {
        if (n[i] < 0 || old[i] < 0 || (int64_t)old[i] + n[i] > INT32_MAX) {
          bad = true;                                    // such a request brings nothing
          n[i] = 0;
          old[i] = old[i] < 0 ? 0 : old[i];
        }
        need[i] = pages(a, old[i] + n[i]) - pages(a, old[i]);
      }
      ts += n[i];
      ps += need[i];
    }
    const int64_t ti = warp_incl_sum(ts, lane), pi = warp_incl_sum(ps, lane);
    __syncthreads();                                     // the step before has read s_tok and s_pg
    if (lane == 31) {
      s_tok[wid] = ti;
      s_pg[wid] = pi;
    }
    __syncthreads();
    int64_t tb = tok + ti - ts, pb = pg + pi - ps;       // before this thread's requests
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < wid) {
        tb += s_tok[w];
        pb += s_pg[w];
      }
      tok += s_tok[w];
      pg += s_pg[w];
    }
    const bool mine = c % gridDim.x == blockIdx.x;       // this CTA writes these requests' results
#pragma unroll
    for (int i = 0; i < kSlotPer; ++i) {
      const int b = c * kSlotTile + tid * kSlotPer + i;
      if (b < a.B && mine) {
        a.context[b] = old[i] + n[i];
        a.start[b] = clamp_i32(tb);
        if (tb + n[i] > a.max_tokens) bad = true;
      }
      if (n[i] > 0 && tb < t1 && tb + n[i] > t0) {
        const int p = tb > t0 ? (int)(tb - t0) : 0;
        s_head[p] = p;
        s_b[p] = b;
        s_old[p] = old[i];
        s_first[p] = pb;
        s_start[p] = tb;
      }
      tb += n[i];
      pb += need[i];
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.start[a.B] = clamp_i32(tok);
    a.used[0] = clamp_i32(pg);
  }
  __syncthreads();
  // running maximum of the head positions over the tile's tokens
  int h[kSlotPer], m = -1;
#pragma unroll
  for (int i = 0; i < kSlotPer; ++i) {
    m = max(m, s_head[tid * kSlotPer + i]);
    h[i] = m;
  }
  int w = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
    if (lane >= o) w = max(w, y);
  }
  if (lane == 31) s_max[wid] = w;
  int before = __shfl_up_sync(0xFFFFFFFFu, w, 1);
  if (lane == 0) before = -1;
  __syncthreads();
  for (int u = 0; u < wid; ++u) before = max(before, s_max[u]);
#pragma unroll
  for (int i = 0; i < kSlotPer; ++i) s_head[tid * kSlotPer + i] = max(before, h[i]);
  __syncthreads();
  // each token's position and where its block id stands; then all block ids, then all results
  const int32_t* from[kSlotPer];
  int32_t* entry[kSlotPer];
  int32_t pos[kSlotPer], off[kSlotPer];
#pragma unroll
  for (int i = 0; i < kSlotPer; ++i) {
    const int64_t t = t0 + i * kSlotThreads + tid;
    from[i] = nullptr;
    entry[i] = nullptr;
    pos[i] = off[i] = 0;
    if (t < t1 && t < tok) {
      const int p = s_head[i * kSlotThreads + tid];
      const int old = s_old[p];
      pos[i] = old + (int32_t)(t - s_start[p]);
      const int page = div_page(a, pos[i]), have = pages(a, old);
      off[i] = pos[i] - page * a.bs;
      if (page < a.bt_stride) {
        int32_t* e = a.table + (int64_t)s_b[p] * a.bt_stride + page;
        const int64_t f = s_first[p] + (page - have);
        if (page < have) from[i] = e;
        else if (f < a.n_free) from[i] = a.free_blocks + f;
        if (page >= have && off[i] == 0) entry[i] = e;
      }
    }
  }
  int32_t blk[kSlotPer];
#pragma unroll
  for (int i = 0; i < kSlotPer; ++i) blk[i] = from[i] != nullptr ? *from[i] : -1;
#pragma unroll
  for (int i = 0; i < kSlotPer; ++i) {
    const int64_t t = t0 + i * kSlotThreads + tid;
    if (t >= t1) continue;
    if (blk[i] < 0 || blk[i] >= a.num_blocks) {
      blk[i] = -1;
      if (t < tok) bad = true;
    }
    if (entry[i] != nullptr) *entry[i] = blk[i];
    a.slot[t] = blk[i] >= 0 ? (int64_t)blk[i] * a.bs + off[i] : -1;
    a.pos[t] = pos[i];
  }
  if (bad) raise_error(DSA_DEVERR_INDEX);
}

}  // namespace

cudaError_t launch_assign_slots(const int32_t* cached, const int32_t* fresh, int B, int bs, const int32_t* free_blocks,
                                int n_free, int64_t num_blocks, int32_t* table, int64_t bt_stride, int64_t max_tokens,
                                int32_t* context, int32_t* start, int64_t* slot, int32_t* pos, int32_t* used,
                                cudaStream_t stream) {
  const int64_t tiles = (max_tokens + kSlotTile - 1) / kSlotTile;
  SlotArgs a{cached, fresh, B, bs, free_blocks, n_free, num_blocks, table, bt_stride, max_tokens,
             context, start, slot, pos, used, 0, 0};
  uint32_t s = 0;
  while ((uint64_t(1) << s) < (uint64_t)bs) ++s;
  a.shift = 31 + s;
  a.mul = bs == 1 ? 0u : (uint32_t)(((uint64_t(1) << a.shift) + (uint64_t)bs - 1) / (uint64_t)bs);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles > 0 ? tiles : 1));
  cfg.blockDim = dim3(kSlotThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, assign_slots_kernel, a);
  note_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

DSA_DEFINE_TU_ERROR_ACCESSORS(slots)

}  // namespace dsa
