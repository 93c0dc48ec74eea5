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
// so its maximum takes four shuffles and no shared memory.
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

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// The 8 elements of piece v of a row.  VEC: elements 8 v .. 8 v + 7, in 16-byte accesses
// (every pointer, stride and D allow it).  Otherwise the 16 lanes of a group take its 128
// elements in turn, element by element: (v / 16) * 128 + 16 i + v % 16.
template <bool VEC>
__device__ __forceinline__ int elem(int v, int i) {
  return VEC ? 8 * v + i : (v >> 4) * 128 + 16 * i + (v & 15);
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int v, int D, float (&f)[8]) {
  if constexpr (VEC) {
    if (8 * v < D) {
      if constexpr (sizeof(T) == 2) {
        const uint4 w = *reinterpret_cast<const uint4*>(row + 8 * v);
        f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
        f[4] = bf16_lo(w.z), f[5] = bf16_hi(w.z), f[6] = bf16_lo(w.w), f[7] = bf16_hi(w.w);
      } else {
        const float4 a = *reinterpret_cast<const float4*>(row + 8 * v);
        const float4 b = *reinterpret_cast<const float4*>(row + 8 * v + 4);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = elem<VEC>(v, i);
      f[i] = e < D ? (float)row[e] : 0.f;
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int v, int D, const float (&f)[8]) {
  if constexpr (VEC) {
    if (8 * v < D) {
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(row + 8 * v) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                            pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
      } else {
        *reinterpret_cast<float4*>(row + 8 * v) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(row + 8 * v + 4) = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = elem<VEC>(v, i);
      if (e < D) row[e] = (T)f[i];
    }
  }
}

// The smallest power of two >= s (s > 0 and finite): its own bits if the mantissa is zero,
// else the next exponent.
__device__ __forceinline__ float next_pow2_f32(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x7FFFFFu) == 0u ? s : __uint_as_float((u & 0x7F800000u) + 0x800000u);
}

// VPT pieces of 8 elements per thread: piece j of thread t of a row is j * tpr + t.
template <typename T, int VPT, bool VEC>
__global__ void __launch_bounds__(VPT == 4 ? 1024 : 512) add_rmsnorm_e4m3_kernel(const NormArgs a) {
  __shared__ float s_sum[32];
  const int rpc = blockDim.x / a.tpr;                  // rows per CTA
  const int sub = threadIdx.x / a.tpr;
  const int t = threadIdx.x - sub * a.tpr;
  const int64_t row = (int64_t)blockIdx.x * rpc + sub;
  const bool live = row < a.T;
  grid_dependency_wait();
  float r[VPT][8];
  float ss = 0.f;
  if (live) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* res = a.res ? static_cast<const T*>(a.res) + row * a.ldr : nullptr;
    T* ro = a.res_out ? static_cast<T*>(a.res_out) + row * a.ldr : nullptr;
#pragma unroll
    for (int j = 0; j < VPT; ++j) load8<T, VEC>(x, j * a.tpr + t, a.D, r[j]);
    if (res != nullptr) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float f[8];
        load8<T, VEC>(res, j * a.tpr + t, a.D, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[j][i] = (float)(T)(r[j][i] + f[i]);
      }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (ro != nullptr) store8<T, VEC>(ro, j * a.tpr + t, a.D, r[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(r[j][i], r[j][i], ss);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  if (a.tpr > 32) {                                    // the row's warps, summed in their order
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = ss;
    __syncthreads();
    const int w0 = (sub * a.tpr) >> 5, nw = a.tpr >> 5;
    ss = 0.f;
    for (int w = 0; w < nw; ++w) ss += s_sum[w0 + w];
  }
  const float rstd = __frsqrt_rn(__fdiv_rn(ss, (float)a.D) + a.eps);
  const int groups = (a.D + 127) >> 7;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = j * a.tpr + t;
    float g[8];
    load8<float, VEC>(a.gamma, v, a.D, g);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r[j][i] = __fmul_rn(__fmul_rn(r[j][i], rstd), g[i]);
      amax = fmaxf(amax, fabsf(r[j][i]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if (!live) continue;
    if (a.y != nullptr) store8<T, VEC>(static_cast<T*>(a.y) + row * a.ldy, v, a.D, r[j]);
    if (a.codes != nullptr && (v >> 4) < groups) {
      float s = 1.f;
      if (amax > 0.f) {
        s = fmaxf(__fdiv_rn(amax, 448.f), 1.17549435e-38f);
        if (a.pow2) s = next_pow2_f32(s);
      }
      const float inv = __fdiv_rn(1.f, s);
      if ((v & 15) == 0) a.scale[row * groups + (v >> 4)] = s;
      uint8_t* c = a.codes + row * a.ldy;
      uint32_t p[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 q = make_float2(__fmul_rn(r[j][i], inv), __fmul_rn(r[j][i + 1], inv));
        p[i >> 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3) << (8 * (i & 3));
      }
      if constexpr (VEC) {
        if (8 * v < a.D) *reinterpret_cast<uint2*>(c + 8 * v) = make_uint2(p[0], p[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = elem<VEC>(v, i);
          if (e < a.D) c[e] = (uint8_t)(p[i >> 2] >> (8 * (i & 3)));
        }
      }
    }
  }
}

constexpr int kNormMaxD = 32768;           // 1024 threads x 4 pieces of 8

template <typename T, int VPT>
cudaError_t launch_norm(const NormArgs& a, bool vec, int threads, int64_t grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return vec ? cudaLaunchKernelEx(&cfg, add_rmsnorm_e4m3_kernel<T, VPT, true>, a)
             : cudaLaunchKernelEx(&cfg, add_rmsnorm_e4m3_kernel<T, VPT, false>, a);
}

template <typename T>
cudaError_t launch_norm_t(NormArgs a, cudaStream_t stream) {
  const auto al = [](const void* p, uintptr_t n) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % n == 0; };
  const int64_t per16 = 16 / (int64_t)sizeof(T);       // elements per 16 bytes
  const bool vec = a.D % 8 == 0 && al(a.x, 16) && a.ldx % per16 == 0 &&
                   ((a.res == nullptr && a.res_out == nullptr) || (al(a.res, 16) && al(a.res_out, 16) && a.ldr % per16 == 0)) &&
                   al(a.gamma, 16) && al(a.codes, 8) && al(a.y, 16) &&
                   ((a.codes == nullptr && a.y == nullptr) || a.ldy % 8 == 0);
  // pieces of 8 elements, whole groups of 16
  const int pieces = (a.D + 127) / 128 * 16;
  const int vpt = pieces <= 512 ? 1 : (pieces <= 1024 ? 2 : 4);
  a.tpr = ((pieces + vpt - 1) / vpt + 31) / 32 * 32;
  const int rpc = a.tpr >= 256 ? 1 : 256 / a.tpr;
  const int64_t grid = (a.T + rpc - 1) / rpc;
  if (vpt == 1) return launch_norm<T, 1>(a, vec, a.tpr * rpc, grid, stream);
  if (vpt == 2) return launch_norm<T, 2>(a, vec, a.tpr * rpc, grid, stream);
  return launch_norm<T, 4>(a, vec, a.tpr * rpc, grid, stream);
}

}  // namespace

int add_rmsnorm_max_dim() { return kNormMaxD; }

cudaError_t launch_add_rmsnorm_e4m3(const void* x, int64_t ldx, const void* res, int64_t ldr, const float* gamma,
                                    float eps, int64_t T, int D, bool f32, void* res_out, void* y, uint8_t* codes,
                                    int64_t ldy, float* scale, bool pow2, cudaStream_t stream) {
  if (T <= 0) return cudaSuccess;
  NormArgs a{x, ldx, res, ldr, gamma, eps, T, D, res_out, y, codes, ldy, scale, pow2 ? 1 : 0, 0};
  const cudaError_t e = f32 ? launch_norm_t<float>(a, stream) : launch_norm_t<__nv_bfloat16>(a, stream);
  note_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace dsa
