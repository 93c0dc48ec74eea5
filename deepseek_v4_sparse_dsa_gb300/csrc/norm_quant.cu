// Residual addition, RMS norm and E4M3 quantisation of hidden rows (sm_103a): what precedes
// the projections that make the indexer's queries, keys and head weights.
//
//   r = round(x + residual) (the residual stream, held in the input's type)
//   y = r * gamma / sqrt(mean(r^2) + eps)                                     in fp32
//   per 128 elements: scale = max|y| / 448 (1 where all are zero), code = E4M3(y / scale)
//
// HBM-bound: bf16 with a residual moves 7 bytes per element (two reads, the new residual and
// the code), so one pass over the row: its threads keep r in registers between the sum of
// squares and the codes.  A group of 128 belongs to 16 neighbouring lanes, 8 elements each,
// so its maximum takes four shuffles and no shared memory.  Measured: 16384 x 4096 bf16 with a
// residual 79 us = 5.9 TB/s (the copy rate is 6.8), 4096 x 4096 fp32 35 us = 6.3 TB/s, 517 x 4999 fp32 without a
// residual 7.5 us in L2 and 9.1 from memory.  16384 x 1536 bf16 without a residual, 3 bytes per element, takes 24 us =
// 3.1 TB/s, one row 1.9 us (the launch).
#include <atomic>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"

namespace dsa {
namespace {

struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* res;           // nullptr: no residual
  int64_t ldr;
  const float* gamma;
  float eps;
  float inv_d;               // 1 / D
  int64_t T;
  int D;
  void* res_out;             // nullable
  void* y;                   // nullable
  uint8_t* codes;            // nullable
  int64_t ldy;
  float* scale;              // [T, ceil(D / 128)]
  int pow2;
  int tpr;                   // threads per row (a multiple of 32)
};

// The 8 elements of piece v of a row, as stored.  VEC: elements 8 v .. 8 v + 7, in 16-byte accesses
// (every pointer, stride and D allow it).  Otherwise the 16 lanes of a group take its 128
// elements in turn, element by element: (v / 16) * 128 + 16 i + v % 16, so that an instruction's
// accesses are neighbours wherever the row starts.
template <typename T, bool VEC>
struct Piece {
  static constexpr int kWords = (int)sizeof(T) * 2;          // 32-bit words of 8 elements
  uint32_t w[kWords];

  static __device__ __forceinline__ int elem(int v, int i) { return VEC ? 8 * v + i : (v >> 4) * 128 + 16 * i + (v & 15); }

  __device__ __forceinline__ void load(const T* row, int v, int D) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = 0u;
    if constexpr (VEC) {
      if (8 * v < D) {
#pragma unroll
        for (int k = 0; k < kWords; k += 4) {
          const uint4 q = reinterpret_cast<const uint4*>(row + 8 * v)[k / 4];
          w[k] = q.x, w[k + 1] = q.y, w[k + 2] = q.z, w[k + 3] = q.w;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = elem(v, i);
        if (e < D) {
          if constexpr (sizeof(T) == 2) w[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(row)[e] << (16 * (i & 1));
          else w[i] = reinterpret_cast<const uint32_t*>(row)[e];
        }
      }
    }
  }

  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 2) return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    else return __uint_as_float(w[i]);
  }

  // w = round(w + o), each sum rounded once to T.
  __device__ __forceinline__ void add(const Piece& o) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 s = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]),
                                         *reinterpret_cast<const __nv_bfloat162*>(&o.w[k]));
        w[k] = *reinterpret_cast<const uint32_t*>(&s);
      } else {
        w[k] = __float_as_uint(__fadd_rn(__uint_as_float(w[k]), __uint_as_float(o.w[k])));
      }
    }
  }

  // Rounds 8 values to T.
  __device__ __forceinline__ void put(const float (&f)[8]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&p);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(f[k]);
    }
  }

  __device__ __forceinline__ void store(T* row, int v, int D) const {
    if constexpr (VEC) {
      if (8 * v < D) {
#pragma unroll
        for (int k = 0; k < kWords; k += 4)
          reinterpret_cast<uint4*>(row + 8 * v)[k / 4] = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = elem(v, i);
        if (e < D) {
          if constexpr (sizeof(T) == 2) reinterpret_cast<uint16_t*>(row)[e] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
          else reinterpret_cast<uint32_t*>(row)[e] = w[i];
        }
      }
    }
  }
};

// The smallest power of two >= s (s > 0, normal): its own bits if the mantissa is zero, else the next
// exponent.
__device__ __forceinline__ float next_pow2_f32(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x7FFFFFu) == 0u ? s : __uint_as_float((u & 0x7F800000u) + 0x800000u);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// VPT pieces of 8 elements per thread: piece j of thread t of a row is j * tpr + t.  A CTA walks the rows
// with a stride of the grid; in 16-byte accesses with one or two pieces the next row's loads are in flight
// while this one is worked on, and gamma stays in registers.  Four pieces leave no room for either.
// Element-wise accesses need the registers for more warps (4096 x 4097 bf16: 79 us with the next row in
// flight, 38 us without); gamma and the residual are loaded with x where they fit (bf16; fp32 517 x 4999
// 6.2 us without, 7.9 us with).  bf16 rows are held to 64 registers (8192 x 7168: 88 -> 76 us), fp32 rows lose by that
// (4096 x 4096: 35 -> 43 us; one piece a thread, held to 64, 128 x 4096: 2.2 -> 3.1 us).  At 64 registers the two-piece
// bf16 kernel spills 36 bytes, the four-piece fp32 kernels 8 and, element by element, 92.  The next launch is
// let in at the start: after the first loads a chain of norm and three products takes 16.5 us for one token, not 15.3.
template <typename T, int VPT, bool VEC>
constexpr int kNormThreads = VEC && sizeof(T) == 4 && VPT < 4 ? (VPT == 2 ? 512 : 768) : 1024;   // at most
template <typename T, int VPT, bool VEC>
__global__ void __launch_bounds__(kNormThreads<T, VPT, VEC>)
    add_rmsnorm_e4m3_kernel(const NormArgs a) {
  using P = Piece<T, VEC>;
  __shared__ float s_sum[2][32];
  const int tpr = a.tpr;
  const int rpc = blockDim.x / tpr;                    // rows per CTA
  const int sub = threadIdx.x / tpr;
  const int t = threadIdx.x - sub * tpr;
  const int groups = (a.D + 127) >> 7;
  const int64_t step = (int64_t)gridDim.x * rpc;
  int64_t row = (int64_t)blockIdx.x * rpc + sub;
  grid_launch_dependents();
  grid_dependency_wait();
  constexpr bool kAhead = VEC && VPT <= 2;
  constexpr bool kAll = VPT <= 2 && (VEC || sizeof(T) == 2);   // gamma and the residual's pieces are held too
  Piece<float, VEC> gm[kAll ? VPT : 1];
  P x[VPT], res[kAll ? VPT : 1];
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = j * tpr + t, D = r < a.T ? a.D : 0;    // nothing past the last row
      x[j].load(static_cast<const T*>(a.x) + r * a.ldx, v, D);
      if (kAll && a.res != nullptr) res[j].load(static_cast<const T*>(a.res) + r * a.ldr, v, D);
    }
  };
  fetch(row);
  if constexpr (kAll) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      gm[j].load(a.gamma, j * tpr + t, a.D);
    }
  }
  for (int it = 0; row - sub < a.T; row += step, it ^= 1) {
    const bool live = row < a.T;
    float r[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (a.res != nullptr) {
        if constexpr (!kAll)
          res[0].load(static_cast<const T*>(a.res) + row * a.ldr, j * tpr + t, live ? a.D : 0);
        x[j].add(res[kAll ? j : 0]);
      }
      if (a.res_out != nullptr && live) x[j].store(static_cast<T*>(a.res_out) + row * a.ldr, j * tpr + t, a.D);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[j][i] = x[j].get(i);
        ss = fmaf(r[j][i], r[j][i], ss);
      }
    }
    if (kAhead && row + step - sub < a.T) fetch(row + step);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (tpr > 32) {                                    // the row's warps, summed in their order
      if ((threadIdx.x & 31) == 0) s_sum[it][threadIdx.x >> 5] = ss;
      __syncthreads();                                 // the other half is free: all have passed the last one
      const int w0 = (sub * tpr) >> 5, nw = tpr >> 5;
      ss = 0.f;
      for (int w = 0; w < nw; ++w) ss += s_sum[it][w0 + w];
    }
    // A sum past fp32 gives rstd 0, as an infinity does: a second, scaled sum for such rows costs the others 2 to 18 %.
    const float rstd = rsqrtf(fmaf(ss, a.inv_d, a.eps));
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = j * tpr + t;
      if constexpr (!kAll) {
        gm[0].load(a.gamma, v, a.D);
      }
      float amax = 0.f;                                // of r * gamma: the row's 1 / rms is a common factor
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[j][i] = __fmul_rn(r[j][i], gm[kAll ? j : 0].get(i));
        amax = fmaxf(amax, fabsf(r[j][i]));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
      if (!live) continue;
      if (a.y != nullptr) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(r[j][i], rstd);
        P y;
        y.put(f);
        y.store(static_cast<T*>(a.y) + row * a.ldy, v, a.D);
      }
      if (a.codes != nullptr) {
        // scale = amax |y| / 448; code = E4M3(y / scale) with y / scale = (r gamma) (448 / amax |r gamma|),
        // one rounding less than by way of y.  Where the scale is a power of two or clamped, or 448 / amax may pass fp32,
        // y comes first and then y / scale: 1 / scale is at most 2^126, while rstd / scale overflows for tiny groups.
        // Each way packs its own codes where a thread has several pieces: r changed in place by one of them costs
        // registers there (16384 x 4096 79 -> 83 us; with one piece 16384 x 128 5.7 us, 5.9 packed apart).
        constexpr bool kApart = VPT > 1;
        constexpr float kMin = 1.17549435e-38f;
        float s = __fmul_rn(__fmul_rn(amax, rstd), 1.f / 448.f), f;
        const auto put_scale = [&] {
          if ((v & 15) == 0 && (v >> 4) < groups) a.scale[row * groups + (v >> 4)] = s;
        };
        uint32_t p[2] = {0u, 0u};
        const auto pack = [&](auto q) {
          if (VEC) put_scale();
#pragma unroll
          for (int i = 0; i < 8; i += 2)
            p[i >> 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q(r[j][i]), q(r[j][i + 1])), __NV_SATFINITE, __NV_E4M3)
                         << (8 * (i & 3));
        };
        if (amax >= 1e-30f && amax <= 1e30f && s >= kMin && !a.pow2) {
          const float r0 = rcp_approx(amax);           // and one Newton step on the quotient: half an ulp
          f = __fmul_rn(448.f, r0);
          f = fmaf(fmaf(-amax, f, 448.f), r0, f);
          if (kApart) pack([&](float z) { return __fmul_rn(z, f); });
        } else {
          if (amax > 0.f && amax < INFINITY && rstd > 0.f) {
            if (s < kMin) s = kMin;
            if (a.pow2) s = next_pow2_f32(s);
            f = __fdiv_rn(1.f, s);
          } else {                                     // zeros, or a row with an infinity (rstd 0) or a NaN, whose codes
            s = 1.f;                                   // are NaN: infinity times 0, NaN times anything
            f = 0.f;
          }
          if (kApart) {
            pack([&](float z) { return __fmul_rn(__fmul_rn(z, rstd), f); });
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[j][i] = __fmul_rn(r[j][i], rstd);
          }
        }
        if (!kApart) pack([&](float z) { return __fmul_rn(z, f); });
        if (!VEC) put_scale();                         // 517 x 4999 fp32: 7.6 us, 8.1 with the scale stored first
        uint8_t* c = a.codes + row * a.ldy;
        if constexpr (VEC) {
          if (8 * v < a.D) *reinterpret_cast<uint2*>(c + 8 * v) = make_uint2(p[0], p[1]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = P::elem(v, i);
            if (e < a.D) c[e] = (uint8_t)(p[i >> 2] >> (8 * (i & 3)));
          }
        }
      }
    }
    if (!kAhead && row + step - sub < a.T) fetch(row + step);
  }
}

constexpr int kNormMaxD = 32768;           // 1024 threads x 4 pieces of 8

template <typename T, int VPT, bool VEC>
cudaError_t launch_norm(const NormArgs& a, int threads, int rpc, int num_sms, cudaStream_t stream) {
  auto* kernel = add_rmsnorm_e4m3_kernel<T, VPT, VEC>;
  // CTAs of this size that an SM holds (asked once per size: every device here is the same)
  static std::atomic<int> held[33];
  int per_sm = held[threads / 32].load(std::memory_order_relaxed);
  if (per_sm == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) per_sm = 1;
    held[threads / 32].store(per_sm, std::memory_order_relaxed);
  }
  const int64_t ctas = (a.T + rpc - 1) / rpc, most = (int64_t)num_sms * per_sm;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(ctas < most ? ctas : most));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, bool VEC>
cudaError_t launch_norm_v(NormArgs a, int num_sms, cudaStream_t stream) {
  // Pieces of 8 elements, whole groups of 16.  A row takes as many threads as it has pieces, or half or a
  // quarter as many: with two pieces a thread there is more in flight per thread and a batch of many
  // rows streams better, unless one warp holds the row anyway (16384 x 128: 7.4 us with two, 4.4 with one);
  // few rows are quickest with one piece a thread (64 x 7168 bf16: 2.5 us, with two 3.8; 304 x 5120: 3.3 and 4.4).
  // Above 768 pieces an SM holds one such row, so that is for a row per SM at most (304 x 7001: 6.5 us with
  // one, 5.6 with two), and fp32 pieces of 32 bytes gain nothing by it (64 x 8192: 3.5 and 3.3).
  const int pieces = (a.D + 127) / 128 * 16;
  const bool wide = pieces > 768;
  const int64_t few = wide ? num_sms : 2 * (int64_t)num_sms;       // rows
  int vpt = pieces <= 32 || (a.T <= few && !(wide && VEC && sizeof(T) == 4)) ? 1 : 2;
  // Rows of more than 1024 pieces: two a thread for a row per SM at most (64 x 8454 bf16: 4.1 us, with four 7.0), and
  // for 16-byte rows with a residual of more than 96 MiB, which the 129 MB L2 cannot keep from the call before, where
  // the next row's loads count: 1300 x 12288 24.9 and 33.2 us, 1800 x 10240 28.8 and 31.0, 4000 x 12288 68 and 89
  // (without a residual 56 and 51).  Below it what lies in L2 goes either way: 600 x 16384 13.3 and 11.5 us, 1200 x
  // 10240 18.0 and 16.8, but 1000 x 12288 18.0 and 20.8; from memory two would win there too (1200 x 10240 20.2 and 23.6).
  if (pieces > 1024) {
    const int64_t bytes = a.T * a.D * (int64_t)(sizeof(T) * (2 + (a.res_out != nullptr) + (a.y != nullptr)) + 1);
    const bool streams = VEC && a.res != nullptr && bytes > (int64_t)96 << 20;
    vpt = pieces <= 2048 && !(VEC && sizeof(T) == 4) && (a.T <= num_sms || streams) ? 2 : 4;
  }
  a.tpr = ((pieces + vpt - 1) / vpt + 31) / 32 * 32;
  const int rpc = a.tpr >= 256 ? 1 : 256 / a.tpr;
  if (vpt == 1) return launch_norm<T, 1, VEC>(a, a.tpr * rpc, rpc, num_sms, stream);
  if (vpt == 2) return launch_norm<T, 2, VEC>(a, a.tpr * rpc, rpc, num_sms, stream);
  return launch_norm<T, 4, VEC>(a, a.tpr * rpc, rpc, num_sms, stream);
}

template <typename T>
cudaError_t launch_norm_t(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const auto al = [](const void* p, uintptr_t n) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % n == 0; };
  const int64_t per16 = 16 / (int64_t)sizeof(T);       // elements per 16 bytes
  const bool vec = a.D % 8 == 0 && al(a.x, 16) && a.ldx % per16 == 0 &&
                   ((a.res == nullptr && a.res_out == nullptr) || (al(a.res, 16) && al(a.res_out, 16) && a.ldr % per16 == 0)) &&
                   al(a.gamma, 16) && al(a.codes, 8) && al(a.y, 16) &&
                   ((a.codes == nullptr && a.y == nullptr) || a.ldy % 8 == 0);
  return vec ? launch_norm_v<T, true>(a, num_sms, stream) : launch_norm_v<T, false>(a, num_sms, stream);
}

}  // namespace

int add_rmsnorm_max_dim() { return kNormMaxD; }

cudaError_t launch_add_rmsnorm_e4m3(const void* x, int64_t ldx, const void* res, int64_t ldr, const float* gamma,
                                    float eps, int64_t T, int D, bool f32, void* res_out, void* y, uint8_t* codes,
                                    int64_t ldy, float* scale, bool pow2, int num_sms, cudaStream_t stream) {
  if (T <= 0) return cudaSuccess;
  NormArgs a{x, ldx, res, ldr, gamma, eps, 1.f / (float)D, T, D, res_out, y, codes, ldy, scale, pow2 ? 1 : 0, 0};
  const cudaError_t e = f32 ? launch_norm_t<float>(a, num_sms, stream) : launch_norm_t<__nv_bfloat16>(a, num_sms, stream);
  note_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace dsa
