// Product of E4M3 rows with E4M3 weights under block scales (sm_103a): the projections that
// make the indexer's queries, keys and head weights.
//
//   out[m, n] = sum_kb sa[m, kb] sw[n / 128, kb] sum_{k in block kb} a[m, k] w[n, k]
//
// Each block of 128 along K is one tcgen05 product into its own TMEM accumulator; the
// epilogue warps multiply it by its two scales and add it to fp32 registers while the next
// block's product runs.
//
// Weight rows are the MMA's M (128 rows: one weight scale per tile and block), BT tokens its N,
// so a decode batch of a few tokens pads to 16 columns instead of 128 rows.  A cluster of S CTAs
// shares a tile, each with its part of K; the parts are added in the order of K through
// distributed shared memory, so that a product with few tiles still streams its weights on
// every SM, and the result does not depend on timing.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "launch.h"

namespace dsa {
namespace {

constexpr int kBlk = 128;                    // K per block, weight rows per tile
constexpr int kGemmThreads = 192;            // producer warp, MMA warp, four epilogue warps
constexpr int kScaleChunk = 16;              // K blocks whose scales are staged at a time
constexpr int kMaxStages = 12;

struct GemmArgs {
  const float* a_scale;                      // [M, G]
  const float* w_scale;                      // [ceil(N / 128), G]
  int64_t M;
  int N;
  int G;                                     // ceil(K / 128)
  void* out;
  int64_t ldo;
  int out_f32;
  int split;                                 // CTAs per tile (the cluster)
  int stages;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t map_peer(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// NC consecutive 32-bit columns of the thread's own TMEM lane (completed by tcgen05.wait::ld).
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

__device__ __forceinline__ void store_out(const GemmArgs& g, int64_t m, int n, float v) {
  if (g.out_f32) static_cast<float*>(g.out)[m * g.ldo + n] = v;
  else static_cast<__nv_bfloat16*>(g.out)[m * g.ldo + n] = __float2bfloat16_rn(v);
}

// Shared memory, from a 1024-byte aligned base: the stages (weights 16 KB, tokens BT * 128
// bytes each), the staged scales [kScaleChunk][BT], the barriers and flags.  The partial sums
// [BT][128] of a split tile reuse the stages once every product has completed.
template <int BT>
__host__ __device__ constexpr uint32_t stage_bytes() { return 16384u + (uint32_t)BT * 128u; }

template <int BT>
size_t gemm_smem(int stages) {
  return 1024 + (size_t)stages * stage_bytes<BT>() + kScaleChunk * BT * 4 + (2 * kMaxStages + 8) * 8 + 16;
}

template <int BT>
__global__ void __launch_bounds__(kGemmThreads) gemm_e4m3_kernel(const __grid_constant__ CUtensorMap tma,
                                                                 const __grid_constant__ CUtensorMap tmw,
                                                                 const GemmArgs g) {
  constexpr uint32_t kStage = stage_bytes<BT>();
  constexpr int kBufs = BT <= 64 ? 4 : 2;                    // TMEM accumulators
  constexpr uint32_t kCols = BT * kBufs < 32 ? 32 : BT * kBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int S = g.split, stages = g.stages;
  float* sc = reinterpret_cast<float*>(sm + (size_t)stages * kStage);
  const uint32_t bars = smem_u32(sc + kScaleChunk * BT);
  int* flags = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(sc + kScaleChunk * BT) + (2 * kMaxStages + 8) * 8);
  volatile int* abort_flag = flags;                          // [0] abort, [1] TMEM base
  auto full = [&](int s) { return bars + 8u * (uint32_t)s; };
  auto empty = [&](int s) { return bars + 8u * (uint32_t)(kMaxStages + s); };
  auto afull = [&](int b) { return bars + 8u * (uint32_t)(2 * kMaxStages + b); };
  auto aempty = [&](int b) { return bars + 8u * (uint32_t)(2 * kMaxStages + 4 + b); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ntiles = (g.N + kBlk - 1) / kBlk;
  const int rank = (int)(blockIdx.x % (unsigned)S);          // = the CTA's rank in its cluster
  const int64_t tile = blockIdx.x / (unsigned)S;
  const int nt = (int)(tile % ntiles);
  const int64_t m0 = tile / ntiles * BT;
  const int mv = g.M - m0 < BT ? (int)(g.M - m0) : BT;       // tokens of this tile
  const int kb0 = (int)((int64_t)g.G * rank / S);
  const int nkb = (int)((int64_t)g.G * (rank + 1) / S) - kb0;
  const unsigned long long limit = wait_limit_ns();

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(afull(b), 1);
      mbar_init(aempty(b), 4);
    }
    flags[0] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&tma);
    tma_prefetch_desc(&tmw);
  }
  if (warp == 1) tmem_alloc(smem_u32(flags + 1), kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)flags[1];
  grid_dependency_wait();

  float acc[BT];
#pragma unroll
  for (int i = 0; i < BT; ++i) acc[i] = 0.f;

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
  } else if (warp == 1) {
    // ================================ MMA issue ================================
    if (lane == 0) {
      constexpr uint32_t kIdesc = idesc_e4m3(128, BT);
      int s = 0, b = 0;
      uint32_t ph = 0, aph = 1;
      bool ok = true;
      int last = -1;
      for (int i = 0; i < nkb; ++i) {
        if (!(ok = mbar_wait(aempty(b), aph, limit, abort_flag) && mbar_wait(full(s), ph, limit, abort_flag))) break;
        tc_fence_after();
        const uint32_t wa = smem_u32(sm) + (uint32_t)s * kStage;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_e4m3(tmem + (uint32_t)(b * BT), smem_desc_sw128(wa + 32u * kk), smem_desc_sw128(wa + 16384u + 32u * kk),
                   kIdesc, kk > 0 ? 1u : 0u);
        mma_commit(empty(s));
        mma_commit(afull(b));
        last = i;
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
        if (++b == kBufs) {
          b = 0;
          aph ^= 1u;
        }
      }
      if (!ok) {
        raise_error(DSA_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      // the last product issued has completed before TMEM is freed or the stages are reused
      if (last >= 0) mbar_wait(afull(last % kBufs), (uint32_t)(last / kBufs) & 1u, kCleanupWaitNs, nullptr);
    }
    __syncwarp();
  } else {
    // ================================ epilogue ================================
    const int gt = threadIdx.x - 64;
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const float* wsc = g.w_scale + (int64_t)nt * g.G + kb0;
    bool ok = true;
    int b = 0;
    uint32_t ph = 0;
    for (int i0 = 0; i0 < nkb; i0 += kScaleChunk) {
      const int nc = min(kScaleChunk, nkb - i0);
      group_sync<128>();                                     // the chunk before has been used
      for (int e = gt; e < BT * kScaleChunk; e += 128) {     // kb fastest: neighbouring addresses
        const int m = e / kScaleChunk, k = e - m * kScaleChunk;
        if (k < nc)
          sc[k * BT + m] = m < mv ? __ldg(g.a_scale + (m0 + m) * g.G + kb0 + i0 + k) * __ldg(wsc + i0 + k) : 0.f;
      }
      group_sync<128>();
      for (int i = 0; i < nc; ++i) {
        if (ok) ok = mbar_wait(afull(b), ph, limit, abort_flag);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok) {
          tc_fence_after();
          const float* f = sc + i * BT;
#pragma unroll
          for (int c = 0; c < BT; c += 16) {
            uint32_t d[16];
            tmem_ld16(tl + (uint32_t)(b * BT + c), d);
            tmem_ld16_wait(d);
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 f4 = *reinterpret_cast<const float4*>(f + c + e);
              acc[c + e] = fmaf(__uint_as_float(d[e]), f4.x, acc[c + e]);
              acc[c + e + 1] = fmaf(__uint_as_float(d[e + 1]), f4.y, acc[c + e + 1]);
              acc[c + e + 2] = fmaf(__uint_as_float(d[e + 2]), f4.z, acc[c + e + 2]);
              acc[c + e + 3] = fmaf(__uint_as_float(d[e + 3]), f4.w, acc[c + e + 3]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(aempty(b));
        }
        if (++b == kBufs) {
          b = 0;
          ph ^= 1u;
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
  if (warp == 1) tmem_dealloc(tmem, kCols);
  const int nrow = 32 * (warp & 3) + lane;                   // the epilogue thread's weight row in the tile
  const int n = nt * kBlk + nrow;
  if (S == 1) {
    if (warp >= 2 && n < g.N) {
#pragma unroll
      for (int m = 0; m < BT; ++m)
        if (m < mv) store_out(g, m0 + m, n, acc[m]);
    }
    return;
  }
  // Split tile: each CTA leaves its part [BT][128] in its own shared memory, CTA r adds up the
  // tokens r, r + S, ... from all parts in rank order.  Every thread passes both cluster
  // barriers once; the second keeps each CTA's memory alive until its peers have read it.
  float* part = reinterpret_cast<float*>(sm);
  if (warp >= 2) {
#pragma unroll
    for (int m = 0; m < BT; ++m)
      if (m < mv) part[m * kBlk + nrow] = acc[m];
  }
  cluster_sync();
  if (warp >= 2 && n < g.N) {
    for (int m = rank; m < mv; m += S) {
      float v = 0.f;
      for (int r = 0; r < S; ++r) v += ld_cluster_f32(map_peer(smem_u32(part + m * kBlk + nrow), (uint32_t)r));
      store_out(g, m0 + m, n, v);
    }
  }
  cluster_sync();
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

template <int BT>
cudaError_t launch_bt(const void* a, int64_t lda, const void* w, int64_t ldw, int64_t K, GemmArgs g, int num_sms,
                      cudaStream_t stream) {
  CUtensorMap tma, tmw;
  if (!make_map(&tma, a, K, g.M, lda, BT) || !make_map(&tmw, w, K, g.N, ldw, kBlk)) return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)((g.N + kBlk - 1) / kBlk) * ((g.M + BT - 1) / BT);
  // split K over a cluster while the tiles leave SMs idle and each part keeps two blocks
  int S = 1;
  while (S < 8 && tiles * S * 2 <= num_sms && 4 * S <= g.G) S *= 2;
  g.split = S;
  const int nkb = (g.G + S - 1) / S;
  int st = 8;
  if (BT == 128) st = 6;
  if (st > nkb) st = nkb < 2 ? 2 : nkb;
  // the partial sums reuse the stages
  while (S > 1 && (size_t)st * stage_bytes<BT>() < (size_t)BT * kBlk * 4) ++st;
  g.stages = st;
  const size_t smem = gemm_smem<BT>(st);
  cudaError_t e = cudaFuncSetAttribute(gemm_e4m3_kernel<BT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * S));
  cfg.blockDim = dim3(kGemmThreads);
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

}  // namespace

cudaError_t launch_gemm_e4m3(const uint8_t* a, int64_t lda, const float* a_scale, const uint8_t* w, int64_t ldw,
                             const float* w_scale, int64_t M, int N, int K, void* out, int64_t ldo, bool out_f32,
                             int num_sms, cudaStream_t stream) {
  if (M <= 0 || N <= 0) return cudaSuccess;
  GemmArgs g{a_scale, w_scale, M, N, (K + kBlk - 1) / kBlk, out, ldo, out_f32 ? 1 : 0, 1, 2};
  cudaError_t e;
  if (M <= 16) e = launch_bt<16>(a, lda, w, ldw, K, g, num_sms, stream);
  else if (M <= 32) e = launch_bt<32>(a, lda, w, ldw, K, g, num_sms, stream);
  else if (M <= 64) e = launch_bt<64>(a, lda, w, ldw, K, g, num_sms, stream);
  else e = launch_bt<128>(a, lda, w, ldw, K, g, num_sms, stream);
  note_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

DSA_DEFINE_TU_ERROR_ACCESSORS(gemm)

}  // namespace dsa
