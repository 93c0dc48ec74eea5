// Product of E4M3 rows with E4M3 weights under block scales (sm_103a): the projections that
// make the indexer's queries, keys and head weights.
//
//   out[m, n] = sum_kb sa[m, kb] sw[n / 128, kb] sum_{k in block kb} a[m, k] w[n, k]
//
// Each block of 128 along K is one tcgen05 product into its own TMEM accumulator; the epilogue warps
// multiply it by its two scales and add it to fp32 registers while the next block's product runs (the
// scales are any fp32 values, so they cannot ride along in the block-scaled MMA).
//
// Few tokens are bound by the weights' stream from memory, many by the way of a block's sums out of TMEM and,
// behind that, by the board's power; what lies between, by the fixed costs of a launch.  Two kernels:
//  * gemm_e4m3_kernel: tiles of 128 weight rows x 16, 32 or 128 tokens.  A cluster of up to 8 CTAs shares a
//    tile, each with its part of K, so that a product with few tiles still streams its weights on every
//    SM; the parts are added in the order of K through distributed shared memory, so the result does
//    not depend on timing and there is no workspace.
//  * gemm_e4m3_pair_kernel: tiles of 256 x 256 on persistent CTA pairs (cta_group::2).
// Measured on quantised normals, operands in L2 and from memory: 1 x 8192 x 2048 5.1 and 5.9 us, 64 x 8192 x 4096
// 9.3 and 10.4 us, 8192 x 64 x 4096 10.2 and 11.6 us.  8192 x 8192 x 4096: 24 calls 214 us each = 2.6 PFLOP/s, run on
// and on 227 to 233 us = 2.4 PFLOP/s, the board at its power limit.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "launch.h"

namespace dsa {
namespace {

constexpr int kBlk = 128;                    // K per block, weight rows per tile
constexpr int kScaleChunk = 16;              // K blocks whose scales are staged at a time
constexpr int kMaxStages = 12;
constexpr size_t kSmemOne = 232448;          // dynamic shared memory of the one CTA of an SM
constexpr size_t kSmemTwo = 115712;          // of each of two (228 KB per SM, 1 KB reserved per CTA)

struct GemmArgs {
  // The scales are read by plain loads, behind the grid's wait: the kernel may be resident while the one that writes
  // them still runs, so they are not constant over its life, which the read-only path requires.
  const float* a_scale;                      // [M, G]
  const float* w_scale;                      // [ceil(N / 128), G]
  int64_t M;
  int N;
  int G;                                     // ceil(K / 128)
  void* out;
  int64_t ldo;
  int out_f32;
  int split_log2;                            // log2 of the CTAs per tile (the cluster)
  int stages;
  int out_vec;                               // out and its rows are 16-byte aligned
  int out_tma;                               // and end on 16 bytes (a bulk tensor store writes whole 16-byte words)
};

// The wait limit as the host has set it (0: the default); the value is needed only behind the set-up.
__device__ __forceinline__ unsigned long long wait_limit_word() {
  return *(volatile unsigned long long*)&g_wait_limit_ns;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t map_peer(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// Half of a cluster barrier each.  A thread's arrival says that its CTA runs, or that products and copies
// which it has seen complete are done with memory that the peers will write; no generic write is
// announced, so it is relaxed.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// 2-D tiled store of a box in shared memory to (x = inner element, y = row), in the thread's bulk group.
__device__ __forceinline__ void tma_store_2d(const void* tmap, uint32_t src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}

__device__ __forceinline__ void tma_prefetch_l2_2d(const void* tmap, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y)
               : "memory");
}

// 16 consecutive 32-bit columns of the thread's own TMEM lane (completed by the wait).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// 32 consecutive 32-bit columns of the thread's own TMEM lane: issue, then completion of every load
// the thread has issued (the registers count as written only there).
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
        "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
        "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
        "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Four sums as they are, eight rounded to bf16.
template <int kN>
__device__ __forceinline__ uint4 four_f32(const float (&v)[kN], int i) {
  return make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3]));
}
template <int kN>
__device__ __forceinline__ uint4 eight_bf16(const float (&v)[kN], int i) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[i + 2 * e], v[i + 2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store_out(const GemmArgs& g, int64_t at, float v) {
  if (g.out_f32) static_cast<float*>(g.out)[at] = v;
  else static_cast<__nv_bfloat16*>(g.out)[at] = __float2bfloat16_rn(v);
}

// Four consecutive outputs of row m from column n (a multiple of 4), rows 16-byte aligned.
__device__ __forceinline__ void store_out4(const GemmArgs& g, int64_t m, int n, float4 v) {
  const int64_t at = m * g.ldo + n;
  if (n + 4 <= g.N) {
    if (g.out_f32) {
      *reinterpret_cast<float4*>(static_cast<float*>(g.out) + at) = v;
    } else {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(g.out) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    return;
  }
  const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < g.N) store_out(g, at + i, e[i]);
}

// Shapes of the kernel with BT tokens per tile.  Four epilogue warps (one per TMEM lane quarter) take
// up to 32 columns; 128 columns are shared by eight.
template <int BT>
struct FewShape {
  static constexpr int kEpi = BT == 128 ? 256 : 128;         // epilogue threads
  static constexpr int kIssue = BT == 128 ? 2 : 1;           // MMA issuers (warps 1 ..)
  static constexpr int kEpi0 = BT == 128 ? 128 : 64;         // first epilogue thread
  static constexpr int kThreads = kEpi0 + kEpi;
  static constexpr int kCols = BT == 128 ? 64 : BT;          // columns per epilogue warp
  // Up to 32 tokens the weight rows are the MMA's M and the tokens its N (a few tokens pad to 16 columns, not
  // to 128 rows), and an epilogue thread holds one weight row of every token: its factors, one per
  // token and block, are read from shared memory.  Reading 128 of them takes the SM's shared-memory
  // bandwidth longer than a block's products (515 of 940 cycles per block at 256 x 8192 x 4096, 17.7 us
  // against 14.7), so with 128 tokens these are the M and the weight rows the N: a thread holds one token,
  // and one factor per block.  64 tokens per tile, either way, won nowhere.
  static constexpr bool kTok = BT == 128;
  static constexpr int kBufs = 4;                            // TMEM accumulators
  static constexpr uint32_t kTmem = BT * kBufs;              // 64 to 512 columns
  static constexpr uint32_t kStage = 16384u + (uint32_t)BT * 128u;   // weights, tokens
  static constexpr uint32_t kScales = BT == 128 ? 0u : 2u * kScaleChunk * BT * 4u;   // two chunks of staged scales
  // The sums of the CTA's tokens from every part: BT * 512 bytes, apart from the stages, so that a CTA
  // need not wait for its peers' products.  128 tokens' 64 KB, and the CTA's own sums as much again,
  // lie over the stages instead.
  static constexpr bool kOver = BT == 128;
  static constexpr uint32_t kIn = kOver ? 0u : (uint32_t)BT * kBlk * 4u;
  static constexpr size_t smem(int stages) {
    return 1024 + (size_t)stages * kStage + kIn + kScales + (2 * kMaxStages + 8) * 8 + 16;
  }
};

// Shared memory, from a 1024-byte aligned base: the stages, the sums that the CTA adds up, the staged
// scales [2][kScaleChunk][BT], the barriers and flags.
template <int BT>
__global__ void __launch_bounds__(FewShape<BT>::kThreads, BT == 128 ? 1 : 2)
    gemm_e4m3_kernel(const __grid_constant__ CUtensorMap tma, const __grid_constant__ CUtensorMap tmw, const GemmArgs g) {
  using Sh = FewShape<BT>;
  const unsigned long long set_limit = wait_limit_word();    // on its way during the set-up
  constexpr uint32_t kStage = Sh::kStage;
  constexpr int kBufs = Sh::kBufs, kEpi = Sh::kEpi, kCols = Sh::kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int lg = g.split_log2, S = 1 << lg, stages = g.stages;
  uint8_t* in_s = Sh::kOver ? sm + BT * kBlk * 4 : sm + (size_t)stages * kStage;
  const uint32_t in = smem_u32(in_s);
  float* sc = reinterpret_cast<float*>(sm + (size_t)stages * kStage + Sh::kIn);
  uint8_t* ctl = sm + (size_t)stages * kStage + Sh::kIn + Sh::kScales;
  const uint32_t bars = smem_u32(ctl);
  int* flags = reinterpret_cast<int*>(ctl + (2 * kMaxStages + 8) * 8);
  volatile int* abort_flag = flags;                          // [0] abort, [1] TMEM base
  auto full = [&](int s) { return bars + 8u * (uint32_t)s; };
  auto empty = [&](int s) { return bars + 8u * (uint32_t)(kMaxStages + s); };
  auto afull = [&](int b) { return bars + 8u * (uint32_t)(2 * kMaxStages + b); };
  auto aempty = [&](int b) { return bars + 8u * (uint32_t)(2 * kMaxStages + 4 + b); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ntiles = (g.N + kBlk - 1) / kBlk;
  const int rank = (int)(blockIdx.x & (unsigned)(S - 1));         // = the CTA's rank in its cluster
  const int tile = (int)(blockIdx.x >> lg);
  const int nt = tile % ntiles;
  const int64_t m0 = (int64_t)(tile / ntiles) * BT;
  const int mv = g.M - m0 < BT ? (int)(g.M - m0) : BT;       // tokens of this tile
  const int kb0 = (int)((int64_t)g.G * rank / S);
  const int nkb = (int)((int64_t)g.G * (rank + 1) / S) - kb0;

  if (warp == 0) {                                           // a barrier per lane: 2 * kMaxStages + 8 of them
    static_assert(2 * kMaxStages + 2 * kBufs == 32, "a barrier per lane");
    mbar_init(bars + 8u * (uint32_t)lane, lane < 32 - kBufs ? 1u : (uint32_t)(kEpi / 32));
    if (lane == 0) {
      flags[0] = 0;
      tma_prefetch_desc(&tma);
      tma_prefetch_desc(&tmw);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (S > 1 && !Sh::kOver) cluster_arrive();
  if (warp == 1) tmem_alloc(smem_u32(flags + 1), Sh::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)flags[1];
  const unsigned long long limit = set_limit == 0 ? kDefaultWaitNs : set_limit;
  grid_launch_dependents();                                  // TMEM is held: the next kernel's set-up may begin
  // While the kernel before this one ends, the weights are brought into L2 (only there: what that
  // kernel may still write to them is seen by the loads behind the wait).  1 x 8192 x 2048 6.3 -> 5.7 us; with
  // 128 tokens it costs up to 10 %.
  if (BT <= 32 && warp == 0 && lane < nkb) tma_prefetch_l2_2d(&tmw, (kb0 + lane) * kBlk, nt * kBlk);
  grid_dependency_wait();

  if (warp == 0) {
    // ================================ producer ================================
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 1;
      int i = 0;
      for (; i < nkb; ++i) {
        if (!mbar_wait(empty(s), ph, limit, abort_flag)) break;
        const uint32_t dst = smem_u32(sm) + (uint32_t)s * kStage;
        mbar_arrive_expect_tx(full(s), kStage);
        tma_load_2d(dst, &tmw, full(s), (kb0 + i) * kBlk, nt * kBlk);
        tma_load_2d(dst + 16384u, &tma, full(s), (kb0 + i) * kBlk, (int)m0);
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (i < nkb) {
        raise_error(DSA_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      // every copy issued has landed before the CTA may leave (a stage's last use is complete
      // once its full barrier's phase is)
      const int issued = i;
      for (int k = issued > stages ? issued - stages : 0; k < issued; ++k)
        mbar_wait(full(k % stages), (uint32_t)(k / stages) & 1u, kCleanupWaitNs, nullptr);
    }
    __syncwarp();
  } else if (warp <= Sh::kIssue) {
    // ================================ MMA issue ================================
    // With 128 tokens a block's products take the tensor core 256 cycles, less than a thread needs
    // for its waits, products and signals: two issuers take the blocks in turn.
    if (lane == 0) {
      constexpr uint32_t kIdesc = idesc_e4m3(128, BT);
      constexpr int kIssue = Sh::kIssue;
      int i = warp - 1, s = i, b = i;
      uint32_t ph = 0, aph = 1;
      for (; i < nkb; i += kIssue) {
        if (!(mbar_wait(aempty(b), aph, limit, abort_flag) && mbar_wait(full(s), ph, limit, abort_flag))) break;
        tc_fence_after();
        const uint32_t wa = smem_u32(sm) + (uint32_t)s * kStage, ta = wa + 16384u;
        const uint32_t ra = Sh::kTok ? ta : wa, ca = Sh::kTok ? wa : ta;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_e4m3(tmem + (uint32_t)(b * BT), smem_desc_sw128(ra + 32u * kk), smem_desc_sw128(ca + 32u * kk), kIdesc,
                   kk > 0 ? 1u : 0u);
        mma_commit(empty(s));
        mma_commit(afull(b));
        if ((s += kIssue) >= stages) {
          s -= stages;
          ph ^= 1u;
        }
        if ((b += kIssue) >= kBufs) {
          b -= kBufs;
          aph ^= 1u;
        }
      }
      if (i < nkb) {
        raise_error(DSA_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      // its last product has completed before TMEM is freed
      const int last = i - kIssue;
      if (last >= 0) mbar_wait(afull(last % kBufs), (uint32_t)(last / kBufs) & 1u, kCleanupWaitNs, nullptr);
    }
    __syncwarp();
  }

  const int gt = threadIdx.x - Sh::kEpi0;                          // epilogue thread
  const int row = 32 * (warp & 3) + lane;                    // its weight row (kTok: token) in the tile
  const int c0 = kCols * (gt >> 7);                          // and its first token (kTok: weight row)
  float acc[kCols];
  if (gt >= 0) {
    // ================================ epilogue ================================
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)c0;
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
    bool ok = true;
    int b = 0;
    uint32_t ph = 0;
    const float* ws = g.w_scale + (int64_t)nt * g.G + kb0;
    // waits for a block's accumulator, reads the warp's columns and hands it back
    auto take = [&](uint32_t (&d)[kCols]) {
      if (ok) ok = mbar_wait(afull(b), ph, limit, abort_flag);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (ok) {
        tc_fence_after();
        const uint32_t from = tl + (uint32_t)(b * BT);
        if constexpr (kCols == 16) {
          tmem_ld16(from, d);
          tmem_ld16_wait(d);
        } else if constexpr (kCols == 32) {
          tmem_ld32_issue(from, d);
          tmem_ld32_wait(d);
        } else {
          tmem_ld64_issue(from, d);
          tmem_ld64_wait(d);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(aempty(b));
      }
      if (++b == kBufs) {
        b = 0;
        ph ^= 1u;
      }
    };
    if constexpr (Sh::kTok) {
      // the token's factor of block i, and of the two blocks after it in flight
      const float* as = g.a_scale + (m0 + min(row, mv - 1)) * g.G + kb0;
      float a0 = as[0], w0 = ws[0], a1 = as[min(1, nkb - 1)], w1 = ws[min(1, nkb - 1)];
      for (int i = 0; i < nkb; ++i) {
        const float f = a0 * w0;
        const int kn = min(i + 2, nkb - 1);
        a0 = a1, w0 = w1;
        a1 = as[kn];
        w1 = ws[kn];
        uint32_t d[kCols];
        take(d);
        if (!ok) break;
#pragma unroll
        for (int e = 0; e < kCols; ++e) acc[e] = fmaf(__uint_as_float(d[e]), f, acc[e]);
      }
    } else {
      // Factors of kScaleChunk blocks at a time, both scales multiplied: thread gt fetches block
      // gt % kScaleChunk of every (kEpi / kScaleChunk)-th token (neighbouring addresses), one chunk
      // ahead, and leaves them in the chunk's half of `sc`.
      constexpr int kPer = BT * kScaleChunk / kEpi, kStep = kEpi / kScaleChunk;
      const int sk = gt % kScaleChunk, sm0 = gt / kScaleChunk;
      const float* as = g.a_scale + m0 * g.G + kb0;
      float pa[kPer], pw;
      auto fetch = [&](int i0) {
        pw = i0 + sk < nkb ? ws[i0 + sk] : 0.f;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
          const int m = sm0 + u * kStep;
          pa[u] = (m < mv && i0 + sk < nkb) ? as[(int64_t)m * g.G + i0 + sk] : 0.f;
        }
      };
      fetch(0);
      for (int i0 = 0, half = 0; i0 < nkb; i0 += kScaleChunk, half ^= 1) {
        float* dst = sc + half * kScaleChunk * BT;
#pragma unroll
        for (int u = 0; u < kPer; ++u) dst[sk * BT + sm0 + u * kStep] = pa[u] * pw;
        group_sync<kEpi>();                                  // the other half is free once all have passed here
        if (i0 + kScaleChunk < nkb) fetch(i0 + kScaleChunk);
        const int nc = min(kScaleChunk, nkb - i0);
        for (int i = 0; i < nc; ++i) {
          uint32_t d[kCols];
          take(d);
          if (!ok) continue;                                 // every warp still passes the chunks' barriers
          const float4* f = reinterpret_cast<const float4*>(dst + i * BT + c0);
#pragma unroll
          for (int e = 0; e < kCols; e += 4) {
            const float4 f4 = f[e / 4];
            acc[e] = fmaf(__uint_as_float(d[e]), f4.x, acc[e]);
            acc[e + 1] = fmaf(__uint_as_float(d[e + 1]), f4.y, acc[e + 1]);
            acc[e + 2] = fmaf(__uint_as_float(d[e + 2]), f4.z, acc[e + 2]);
            acc[e + 3] = fmaf(__uint_as_float(d[e + 3]), f4.w, acc[e + 3]);
          }
        }
      }
    }
    if (!ok && lane == 0) {
      raise_error(DSA_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, Sh::kTmem);
  // The sums of token m go to CTA m % S of the cluster, as rows of 128 weight rows' sums: row
  // rank * per + m / S of its `in`.  Behind a cluster barrier each CTA adds its tokens' parts in rank
  // order from its own memory, four neighbouring outputs per thread, and no CTA reads another's.
  // A warp writes whole rows (32 lanes, neighbouring addresses): with the lanes' 16-byte pieces spread
  // over rows and CTAs the writes to the peers took 2.6 us instead of 1.
  const int per = BT >> lg;                                  // tokens of a CTA
  if (S > 1) {                                               // the peers run, and where the sums lie over
    if (Sh::kOver) cluster_arrive();                         // the stages their products are done
    cluster_wait();
  }
  if constexpr (Sh::kTok) {
    // The CTA's own sums first: 16-byte pieces of the token's row, piece p at p ^ (token & 7), so that
    // eight lanes' pieces fall into different banks.
    if (gt >= 0) {
      float4* own = reinterpret_cast<float4*>(sm + 512 * row);
#pragma unroll
      for (int p = 0; p < kCols / 4; ++p)
        own[(c0 / 4 + p) ^ (row & 7)] = make_float4(acc[4 * p], acc[4 * p + 1], acc[4 * p + 2], acc[4 * p + 3]);
      group_sync<kEpi>();
      if (S > 1) {
#pragma unroll 4
        for (int m = gt >> 5; m < mv; m += kEpi / 32) {
          const int r = m & (S - 1);
          const float4 v = reinterpret_cast<const float4*>(sm)[32 * m + lane];
          if (r != rank && nt * kBlk + 4 * (lane ^ (m & 7)) < g.N)
            st_cluster_f32x4(map_peer(in + 512u * (uint32_t)(rank * per + (m >> lg)) + 16u * lane, (uint32_t)r), v);
        }
      }
    }
  } else if (gt >= 0) {
    const uint32_t at = in + 4u * (uint32_t)(rank * per * kBlk + row);
#pragma unroll
    for (int e = 0; e < kCols; ++e) {
      const int m = c0 + e;
      if (m < mv) st_cluster_f32(map_peer(at + 512u * (uint32_t)(m >> lg), (uint32_t)(m & (S - 1))), acc[e]);
    }
  }
  if (S > 1) cluster_sync();
  else __syncthreads();
  if (gt < 0) return;
  constexpr int kRows = kEpi / 32;                           // warps, a row each
  // row of part r of the CTA's token j
  const auto part = [&](int r, int j) { return Sh::kTok && r == rank ? sm + 512 * (rank + S * j) : in_s + 512 * (r * per + j); };
  if (g.out_vec) {
    const int n = nt * kBlk + 4 * lane;
    if (n >= g.N) return;
    constexpr int kFly = 4;                                  // rows in flight per warp
    for (int j0 = gt >> 5; rank + S * j0 < mv; j0 += kRows * kFly) {
      float4 v[kFly];
#pragma unroll
      for (int u = 0; u < kFly; ++u) v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int r = 0; r < S; ++r) {
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
          const int j = j0 + u * kRows, m = rank + S * j;
          if (m < mv) {
            const float4 t = reinterpret_cast<const float4*>(part(r, j))[Sh::kTok ? lane ^ (m & 7) : lane];
            v[u].x += t.x, v[u].y += t.y, v[u].z += t.z, v[u].w += t.w;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        const int m = rank + S * (j0 + u * kRows);
        if (m < mv) store_out4(g, m0 + m, n, v[u]);
      }
    }
  } else {                                                   // rows at any alignment: neighbouring elements
    constexpr int kFly = 4;
    for (int j0 = gt >> 5; rank + S * j0 < mv; j0 += kRows * kFly) {
      float v[kFly][4];
#pragma unroll
      for (int u = 0; u < kFly; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) v[u][q] = 0.f;
      for (int r = 0; r < S; ++r) {
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
          const int j = j0 + u * kRows, m = rank + S * j;
          if (m < mv) {
            const float* from = reinterpret_cast<const float*>(part(r, j));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int c = lane + 32 * q;
              v[u][q] += from[Sh::kTok ? c ^ ((m & 7) << 2) : c];
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        const int m = rank + S * (j0 + u * kRows);
        if (m < mv) {
          const int64_t at = (m0 + m) * g.ldo + nt * kBlk + lane;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (nt * kBlk + lane + 32 * q < g.N) store_out(g, at + 32 * q, v[u][q]);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ many tokens
// A pair of CTAs (one cluster, cta_group::2) owns a tile of 256 tokens x 256 weight rows: each
// CTA holds 128 of the tokens and 128 of the weight rows in shared memory (32 KB per block of
// K), the pair's tensor cores read both, and each CTA's TMEM receives its 128 tokens x 256
// columns.  Tokens are the MMA's M here, so an epilogue thread owns one token: one activation
// scale per block.  Two accumulators of 256 columns fill TMEM: the epilogue adds block kb to its
// registers while block kb + 1 runs.  Warps: producer, two MMA issuers (the even CTA's), one that
// tells the even CTA that this CTA's copies have landed, eight epilogue warps (128 columns each).
// The pairs walk the tiles in groups of 8 token tiles, so that the tiles in flight share rows.
// Bound by the accumulators' way back to the issuers: 837 cycles per block at 1.8 to 1.9 GHz, where the products alone
// need 512.  Power comes next: 16384 x 8192 x 8192 runs at 2.85 PFLOP/s in a burst, and on and on at 2.6 with 1.39 of
// 1.4 kW and 1.8 GHz; without the sums the products alone reach 3.1 PFLOP/s.
constexpr int kPairThreads = 384;             // warps 0..3: producer, two MMA issuers, forwarder; 4..11: epilogue
constexpr int kPairStages = 5;
constexpr uint32_t kPairStage = 32768u;      // 128 tokens and 128 weight rows of 128 bytes
constexpr uint32_t kPairStaging = 8u * 8192u;   // two blocks of 32 x 128 bytes per epilogue warp
constexpr size_t kPairSmem = 1024 + kPairStages * kPairStage + kPairStaging + 64 * 8;

// Arrives on a barrier of a CTA of the cluster, without the cluster-wide release that makes a thread wait
// for all its memory operations (with it 8192 x 8192 x 4096 took 508 us, without 280).  What it announces is no
// generic write: TMEM reads whose values are in registers, or copies that the thread's own barrier has
// seen land in its CTA's shared memory, which that CTA's tensor core reads.
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ void mma_e4m3_pair(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(
          tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives on the barrier at this offset in both CTAs once every product issued so far is done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

__global__ void __launch_bounds__(kPairThreads, 1) gemm_e4m3_pair_kernel(const __grid_constant__ CUtensorMap tma,
                                                                         const __grid_constant__ CUtensorMap tmw,
                                                                         const __grid_constant__ CUtensorMap tmo,
                                                                         const GemmArgs g) {
  const unsigned long long set_limit = wait_limit_word();    // on its way during the set-up
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t bars = smem_u32(sm + kPairStages * kPairStage + kPairStaging);
  int* flags = reinterpret_cast<int*>(sm + kPairStages * kPairStage + kPairStaging + 60 * 8);
  volatile int* abort_flag = flags;                          // [0] abort, [1] TMEM base
  auto full = [&](int s) { return bars + 8u * (uint32_t)s; };
  auto ready = [&](int s) { return bars + 8u * (uint32_t)(8 + s); };   // even CTA: both CTAs' copies have landed
  auto empty = [&](int s) { return bars + 8u * (uint32_t)(16 + s); };
  auto afull = [&](int b) { return bars + 8u * (uint32_t)(24 + b); };
  auto aempty = [&](int b) { return bars + 8u * (uint32_t)(26 + b); };
  const uint32_t drain = bars + 8u * 28u;                    // both issuers' products and signals are done

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1u;                     // = the CTA's rank in its cluster
  const int pair = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);
  const int mt = (int)((g.M + 255) / 256), nt = (g.N + 255) / 256;
  const int tiles = mt * nt;
  const int G = g.G;

  // token tile and weight tile of tile t: groups of 8 token tiles, tokens fastest
  auto locate = [&](int t, int& m0, int& n0) {
    const int per = 8 * nt;
    const int grp = t / per;
    const int h = min(8, mt - 8 * grp);
    const int r = t - grp * per;
    m0 = (8 * grp + r % h) * 256;
    n0 = r / h * 256;
  };

  if (warp == 0) {                                           // a barrier per lane (full, ready, empty: 8 each; 2 + 2; 1)
    if (lane < 29)
      mbar_init(bars + 8u * (uint32_t)lane, lane == 28 || (lane >= 8 && lane < 16) ? 2u : (lane >= 26 ? 16u : 1u));
    if (lane == 0) {
      flags[0] = 0;
      tma_prefetch_desc(&tma);
      tma_prefetch_desc(&tmw);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(flags + 1)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)flags[1];
  const unsigned long long limit = set_limit == 0 ? kDefaultWaitNs : set_limit;
  grid_launch_dependents();                                  // TMEM is held: the next kernel's set-up may begin
  grid_dependency_wait();

  // The epilogue's 128 sums, 64 columns in flight and their scales need more than the 168 registers
  // that 12 warps leave each thread: the first four warps hand theirs over
  // (128 x 64 + 256 x 216 <= 384 x 168).
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  if (warp == 0) {
    // ================================ producer ================================
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 1;
      int issued = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += npairs) {
        int m0, n0;
        locate(t, m0, n0);
        for (int kb = 0; kb < G; ++kb) {
          if (!(ok = mbar_wait(empty(s), ph, limit, abort_flag))) break;
          const uint32_t dst = smem_u32(sm) + (uint32_t)s * kPairStage;
          mbar_arrive_expect_tx(full(s), kPairStage);
          tma_load_2d(dst, &tma, full(s), kb * kBlk, m0 + 128 * (int)rank);
          tma_load_2d(dst + 16384u, &tmw, full(s), kb * kBlk, n0 + 128 * (int)rank);
          ++issued;
          if (++s == kPairStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) {
        raise_error(DSA_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      // before the CTA may leave: every copy has landed, and (unless the call was abandoned)
      // the products' last signals to this CTA's stages have arrived
      for (int k = issued > kPairStages ? issued - kPairStages : 0; k < issued; ++k) {
        const int st = k % kPairStages;
        const uint32_t par = (uint32_t)(k / kPairStages) & 1u;
        mbar_wait(full(st), par, kCleanupWaitNs, nullptr);
        if (ok) ok = mbar_wait(empty(st), par, limit, abort_flag);
      }
      // An abandoned call's CTA does not know how many products the pair has issued: their signals reach both CTAs, so
      // neither leaves before the issuers' last one, which follows all others.
      mbar_wait(drain, 0u, kCleanupWaitNs, nullptr);
    }
    __syncwarp();
  } else if (warp < 4) {
    const int n = pair < tiles ? (tiles - pair + npairs - 1) / npairs * G : 0;   // the pair's blocks, over all its tiles
    if (lane == 0 && warp == 3) {
      // ================ tells the MMA issuers that this CTA's copies have landed ================
      int s = 0;
      uint32_t ph = 0;
      for (int k = 0; k < n; ++k) {
        if (!mbar_wait(full(s), ph, limit, abort_flag)) {
          raise_error(DSA_DEVERR_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        arrive_cluster(map_peer(ready(s), 0u));
        if (++s == kPairStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    } else if (lane == 0 && rank == 0) {
      // ================================ MMA issue ================================
      // Warp 1 issues the even blocks, warp 2 the odd ones, each into its own accumulator: a thread
      // is held while the tensor core takes its products, and its waits and signals for the next
      // block run behind the other's products.
      constexpr uint32_t kIdesc = idesc_e4m3(256, 256);
      const int b = warp - 1;
      const uint32_t acc = tmem + 256u * (uint32_t)b;
      const uint64_t desc0 = smem_desc_sw128(smem_u32(sm));
      int s = b, k = b;
      uint32_t ph = 0, aph = 1;
      for (; k < n; k += 2) {
        if (!(mbar_wait(ready(s), ph, limit, abort_flag) && mbar_wait(aempty(b), aph, limit, abort_flag))) break;
        tc_fence_after();
        const uint64_t da = desc0 + (uint64_t)(s * (int)(kPairStage >> 4));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)                       // 32 bytes of K along the rows; the weights 16 KB on
          mma_e4m3_pair(acc, da + 2u * kk, da + 1024u + 2u * kk, kIdesc, kk > 0 ? 1u : 0u);
        mma_commit_pair(empty(s));
        mma_commit_pair(afull(b));
        aph ^= 1u;
        if ((s += 2) >= kPairStages) {
          s -= kPairStages;
          ph ^= 1u;
        }
      }
      if (k < n) {
        raise_error(DSA_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      // the last product has completed before either CTA frees TMEM or leaves
      mma_commit_pair(drain);
      if (k > b) mbar_wait(afull(b), (uint32_t)((k - 2) >> 1) & 1u, kCleanupWaitNs, nullptr);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ================================ epilogue ================================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int half = (warp - 4) >> 2;                        // columns 128 half .. 128 half + 127
    const int quarter = warp & 3;                            // TMEM lanes 32 quarter ..
    const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16) + 128u * (uint32_t)half;
    uint8_t* staging = sm + kPairStages * kPairStage + (uint32_t)(warp - 4) * 8192u;
    const uint32_t aempty0 = map_peer(aempty(0), 0u);
    bool ok = true;
    int b = 0;
    uint32_t ph = 0;
    for (int t = pair; ok && t < tiles; t += npairs) {
      int m0, n0;
      locate(t, m0, n0);
      m0 += 128 * (int)rank + 32 * quarter;                  // the warp's first token
      n0 += 128 * half;                                      // and first column
      const int64_t mrow = min((int64_t)m0 + lane, g.M - 1);
      const int nblk = n0 < g.N ? n0 / kBlk : (g.N - 1) / kBlk;
      const float* as = g.a_scale + mrow * G;
      const float* ws = g.w_scale + (int64_t)nblk * G;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      // scales of block kb, and of the two after it in flight
      float a0 = as[0], w0 = ws[0], a1 = as[min(1, G - 1)], w1 = ws[min(1, G - 1)];
      for (int kb = 0; kb < G; ++kb) {
        const float f = a0 * w0;
        const int kn = min(kb + 2, G - 1);
        a0 = a1, w0 = w1;
        a1 = as[kn];
        w1 = ws[kn];
        ok = mbar_wait(afull(b), ph, limit, abort_flag);
        if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
        tc_fence_after();
        const uint32_t ta = tl + 256u * (uint32_t)b;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t d[64];
          tmem_ld64_issue(ta + 64u * c, d);
          tmem_ld64_wait(d);
          if (c == 1) {                                      // all columns read: the accumulator is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(aempty0 + 8u * (uint32_t)b);
          }
#pragma unroll
          for (int e = 0; e < 64; ++e) acc[64 * c + e] = fmaf(__uint_as_float(d[e]), f, acc[64 * c + e]);
        }
        if ((b ^= 1) == 0) ph ^= 1u;
      }
      if (!ok) break;
      const int rows = g.M - m0 < 32 ? (int)(g.M - m0) : 32;
      if (g.out_tma) {
        // The warp's 32 tokens x 128 columns leave through its two staging blocks, 128 bytes of each row at a
        // time: a thread writes its own row's pieces in the 128-byte swizzle, one lane hands the block to
        // a bulk tensor store (which leaves out what lies past M and N), and the warp goes on.
        auto put = [&](int col0, int block, const uint4 (&v)[8]) {
          uint8_t* stage = staging + 4096 * block;
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");   // the block's last store is read
          __syncwarp();
#pragma unroll
          for (int p = 0; p < 8; ++p) *reinterpret_cast<uint4*>(stage + lane * 128 + ((p ^ (lane & 7)) << 4)) = v[p];
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            if (rows > 0 && col0 < g.N) tma_store_2d(&tmo, smem_u32(stage), col0, m0);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        };
        if (g.out_f32) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 v[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) v[p] = four_f32(acc, 32 * q + 4 * p);
            put(n0 + 32 * q, q & 1, v);
          }
        } else {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint4 v[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) v[p] = eight_bf16(acc, 64 * q + 8 * p);
            put(n0 + 64 * q, q, v);
          }
        }
      } else {
        // Rows at any alignment, through the staging blocks. fp32: a row's 128 columns at a time, every store
        // instruction in one 128-byte line, so that only a row's two ends write part of a 32-byte sector:
        // 241 us at 6732 x 14163 x 1792, where words stored from each 128-byte piece's own start
        // took 264. bf16, whose row has half the sectors, keeps to its pieces (207 us; in whole lines 223,
        // and 280 with the rows' ends stored apart).
        const int cols = g.N > n0 ? min(128, g.N - n0) : 0;
        if (g.out_f32) {
          const uint32_t first = (uint32_t)((reinterpret_cast<uintptr_t>(g.out) >> 2) + (uint64_t)((int64_t)m0 * g.ldo + n0));   // in words
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {                      // 16 rows of 512 bytes
            if ((lane >> 4) == h) {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                *reinterpret_cast<uint4*>(staging + (lane & 15) * 512 + (((q & 24) | ((q ^ lane) & 7)) << 4)) = four_f32(acc, 4 * q);
            }
            __syncwarp();
#pragma unroll 1
            for (int r0 = 0; r0 < 16; r0 += 4) {             // four rows in flight, no branches
              uint32_t x[4][5];
              int c0[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int r = r0 + u;
                const uint32_t at = first + (uint32_t)(16 * h + r) * (uint32_t)g.ldo;
                c0[u] = lane - (int)(at & 31u);
#pragma unroll
                for (int k = 0; k < 5; ++k) {
                  const int c = (c0[u] + 32 * k) & 127, q = c >> 2;
                  x[u][k] = *reinterpret_cast<const uint32_t*>(staging + r * 512 + (((q & 24) | ((q ^ r) & 7)) << 4) + 4 * (c & 3));
                }
              }
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                uint32_t* o = static_cast<uint32_t*>(g.out) + (int64_t)(m0 + 16 * h + r0 + u) * g.ldo + n0 + c0[u];
                const int lim = 16 * h + r0 + u < rows ? cols : 0;
#pragma unroll
                for (int k = 0; k < 5; ++k)
                  if ((unsigned)(c0[u] + 32 * k) < (unsigned)lim) o[32 * k] = x[u][k];
              }
            }
            __syncwarp();
          }
        } else {
          // a bf16 row that starts at 2 mod 4 has its words shifted by one element, and its first and last
          // element apart
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint8_t* stage = staging + 4096 * q;
#pragma unroll
            for (int p = 0; p < 8; ++p)
              *reinterpret_cast<uint4*>(stage + lane * 128 + ((p ^ (lane & 7)) << 4)) = eight_bf16(acc, 64 * q + 8 * p);
            __syncwarp();
            const int lim = min(64, cols - 64 * q);
            constexpr int kFly = 8;
#pragma unroll 1
            for (int r0 = 0; r0 < rows; r0 += kFly) {
              uint32_t w[kFly];
#pragma unroll
              for (int u = 0; u < kFly; ++u)
                w[u] = *reinterpret_cast<const uint32_t*>(stage + (r0 + u) * 128 + (((lane >> 2) ^ ((r0 + u) & 7)) << 4) + 4 * (lane & 3));
#pragma unroll
              for (int u = 0; u < kFly; ++u) {
                uint16_t* o = static_cast<uint16_t*>(g.out) + (int64_t)(m0 + r0 + u) * g.ldo + n0 + 64 * q;
                const bool live = r0 + u < rows;
                const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, w[u], 1);
                const int odd = (int)(reinterpret_cast<uintptr_t>(o) >> 1) & 1, e = 2 * lane + odd;
                const uint32_t x = odd ? __funnelshift_r(w[u], next, 16) : w[u];
                const bool whole = e + 1 < lim;
                if (live && whole) *reinterpret_cast<uint32_t*>(o + e) = x;
                if (live && !whole && e < lim) o[e] = (uint16_t)x;
                if (live && odd && lane == 0 && lim > 0) o[0] = (uint16_t)w[u];
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
    if (!ok && lane == 0) {
      raise_error(DSA_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
  }
  // both CTAs are done with each other's barriers, shared memory and TMEM
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// ------------------------------------------------------------------ host side
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

// Rows of K bytes, `ld` bytes apart; boxes of 128 bytes x box_rows in the 128-byte swizzle.
// What lies past K or past the last row reads as zeros.
bool make_map(CUtensorMap* m, const void* base, int64_t K, int64_t rows, int64_t ld, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {128u, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The result in boxes of 32 rows x 128 bytes, in the 128-byte swizzle.
bool make_out_map(CUtensorMap* m, const GemmArgs& g) {
  auto fn = encode_fn();
  if (!fn) return false;
  const uint32_t es = g.out_f32 ? 4u : 2u;
  const cuuint64_t dims[2] = {(cuuint64_t)g.N, (cuuint64_t)g.M};
  const cuuint64_t strides[1] = {(cuuint64_t)g.ldo * es};
  const cuuint32_t box[2] = {128u / es, 32u};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, g.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.out, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Lets a kernel ask for up to kSmemOne bytes of shared memory on the current device: once per kernel and
// device (`devices` has a bit for each), not on every call.
template <typename K>
cudaError_t allow_smem(K* kernel, std::atomic<uint64_t>& devices) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (devices.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemOne);
  if (e == cudaSuccess) devices.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// log2 of the CTAs that share a tile's K: twice as many while the tiles leave CTA slots free and each part
// keeps two blocks, up to 8.  Clusters of 8 leave SMs of a GPC over, so they may ask for three quarters of
// the slots only (16 clusters of 8, one CTA per SM, ran in two waves: 128 x 2048 x 2048 11.4 us).
int split_log2(int64_t tiles, int G, int64_t slots) {
  int lg = 0;
  while (lg < 3 && (tiles << (lg + 1)) <= (lg == 2 ? slots * 3 / 4 : slots) && (4 << lg) <= G) ++lg;
  return lg;
}

template <int BT>
cudaError_t launch_bt(const void* a, int64_t lda, const void* w, int64_t ldw, int64_t K, GemmArgs g, int num_sms,
                      cudaStream_t stream) {
  CUtensorMap tma, tmw;
  if (!make_map(&tma, a, K, g.M, lda, BT) || !make_map(&tmw, w, K, g.N, ldw, kBlk)) return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)((g.N + kBlk - 1) / kBlk) * ((g.M + BT - 1) / BT);
  const int lg = split_log2(tiles, g.G, (int64_t)num_sms * (BT == 128 ? 1 : 2));   // two CTAs per SM up to 32 tokens
  const int S = 1 << lg;
  g.split_log2 = lg;
  const int nkb = (g.G + S - 1) / S;
  // as many stages as shared memory holds, and no more than there are blocks
  int st = 2;
  const size_t room = BT == 128 ? kSmemOne : kSmemTwo;
  while (st < kMaxStages && st < nkb && FewShape<BT>::smem(st + 1) <= room) ++st;
  if (FewShape<BT>::kOver && S > 1 && st < 4) st = 4;        // 128 KB of sums
  g.stages = st;
  const size_t smem = FewShape<BT>::smem(st);
  static std::atomic<uint64_t> devices{0};
  const cudaError_t e = allow_smem(gemm_e4m3_kernel<BT>, devices);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * S));
  cfg.blockDim = dim3(FewShape<BT>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm_e4m3_kernel<BT>, tma, tmw, g);
}

cudaError_t launch_pair(const void* a, int64_t lda, const void* w, int64_t ldw, int64_t K, const GemmArgs& g,
                        int num_sms, cudaStream_t stream) {
  CUtensorMap tma, tmw, tmo;
  if (!make_map(&tma, a, K, g.M, lda, 128) || !make_map(&tmw, w, K, g.N, ldw, 128)) return cudaErrorInvalidValue;
  if (!g.out_tma) {
    memset(&tmo, 0, sizeof(tmo));                            // rows are stored without it
  } else if (!make_out_map(&tmo, g)) {
    return cudaErrorInvalidValue;
  }
  static std::atomic<uint64_t> devices{0};
  const cudaError_t e = allow_smem(gemm_e4m3_pair_kernel, devices);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((g.M + 255) / 256) * (int64_t)((g.N + 255) / 256);
  const int64_t pairs = tiles < num_sms / 2 ? tiles : num_sms / 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm_e4m3_pair_kernel, tma, tmw, tmo, g);
}

}  // namespace

cudaError_t launch_gemm_e4m3(const uint8_t* a, int64_t lda, const float* a_scale, const uint8_t* w, int64_t ldw,
                             const float* w_scale, int64_t M, int N, int K, void* out, int64_t ldo, bool out_f32,
                             int num_sms, cudaStream_t stream) {
  if (M <= 0 || N <= 0) return cudaSuccess;
  GemmArgs g{a_scale, w_scale, M, N, (K + kBlk - 1) / kBlk, out, ldo, out_f32 ? 1 : 0, 0, 2, 0, 0};
  const int64_t es = out_f32 ? 4 : 2;
  // A single row's stride is any number: no products of it that could overflow.
  g.out_vec = reinterpret_cast<uintptr_t>(out) % 16 == 0 && ldo % (16 / es) == 0 ? 1 : 0;
  g.out_tma = g.out_vec && N * es % 16 == 0 && ldo < ((int64_t)1 << 40) / es ? 1 : 0;
  // Tiles of 128 x 128 that fill the SMs more than once go to the CTA pairs (operands from memory): 512 x 8192 x 4096
  // 19.6 us against 28.8, 130 x 9800 x 4096 19.3 and 23.9, 256 x 9984 x 4096 19.3 and 28.0, 257 x 6500 x 4096 20.8 and
  // 23.7, while at 256 x 8192 x 4096 (one wave) the clusters win (15.0 and 19.0).  The rule does not look at the tokens:
  // up to 128 of them with more than 152 x 128 columns the pairs lose (128 x 19584 x 4096 34.1 us against 30.8, 64 x
  // 24576 x 4096 34.1 and 28.6, 1 x 24576 x 4096 36.6 and 22.0 with 16 tokens).
  // Tiles of 32 tokens pay where those of 128, split over K, leave half the SMs idle (128 x 512 x 8192 7.2 us
  // against 8.5 with 128 tokens, 500 x 128 x 4096 5.6 and 7.1); elsewhere they read the weights too often
  // (333 x 1000 x 1808 7.9 and 7.2 us, 95 x 2816 x 6704 13.8 and 10.5).  Up to 16 tokens 16 columns suffice.
  const int64_t nt = (N + 127) / 128;
  cudaError_t e;
  if ((M + 127) / 128 * nt > num_sms) e = launch_pair(a, lda, w, ldw, K, g, num_sms, stream);
  else if (M <= 16) e = launch_bt<16>(a, lda, w, ldw, K, g, num_sms, stream);
  else if (M <= 32 || ((M + 127) / 128 * nt << split_log2((M + 127) / 128 * nt, g.G, num_sms)) * 2 < num_sms)
    e = launch_bt<32>(a, lda, w, ldw, K, g, num_sms, stream);
  else e = launch_bt<128>(a, lda, w, ldw, K, g, num_sms, stream);
  note_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

DSA_DEFINE_TU_ERROR_ACCESSORS(gemm)

}  // namespace dsa
