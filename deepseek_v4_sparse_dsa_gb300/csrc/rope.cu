// Rotary positions (sm_103a): the cos / sin table, the rotation of heads by it, and the same rotation behind a
// per-head RMS norm with keys and values going to their cache slots.
//
//   table   f_i = base^(-2i / R), i < R / 2, or scaled; angle(p, i) = p f_i
//   rope    (x0, x1) -> (x0 c - x1 s, x0 s + x1 c) for the pairs (2i, 2i + 1) or (i, i + R / 2) of R dims of a head
//   norm    y = x gamma / sqrt(mean(x^2) + eps) over the head's D dims, before the rotation
//
// Sums, norm and rotation are fp32; a result is rounded once, to the rows' type or to the cache's bf16.
//
// All of it streams: each element is read once and written once, the table's rows come from L2.  Measured: rotation of
// 8192 x 64 x 128 in bf16 44 us (92 % of the copy rate), in fp32 82 (97 %); 8192 tokens of 64 query and 8 key and value
// heads with the norm 63 us (79 %; HBM and issue slots together), in halves 60, in fp32 98 (96 %), without it 52 (95 %); a
// table of 1 M positions x 64 51 us (77 %; instructions); one token 3.0 us.
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "launch.h"

namespace dsa {
namespace {

// ------------------------------------------------------------------ table
// An angle is needed modulo a turn only.  With W_i = f_i / 2 pi turns as a 64-bit binary fraction, the product p W_i
// modulo 2^64 is the angle's fraction of a turn, exact but for W's truncation (p 2^-64 turns): far positions lose
// nothing and no 64-bit floating point is needed.  The nearest quarter turn is taken off before the conversion to
// fp32, so that what is left, at most 1/8 turn, keeps 24 significant bits; there the Taylor polynomials of degree 9 and 8
// are within 2.5e-8 of the sine and the cosine (the terms left out: x^11 / 11!, x^10 / 10! at pi / 4).
// Bound by the writes once a pair costs few enough instructions: 1 M positions x 64 took 74 us with sincospi and the
// remainder converted as one 64-bit number.
struct TableArgs {
  uint64_t turn[128];        // f_i / 2 pi in units of 2^-64 turns
  int64_t pos0, n;
  int half;                  // R / 2
  int rows;                  // rows of a block's pass: as many as its threads cover
  float sine[5], cosine[5];  // the polynomials' coefficients times the amplitude, lowest first
  float* out;
};

__device__ __forceinline__ void write_angle(const TableArgs& a, int64_t row, int i, uint64_t phase) {
  const uint32_t high = (uint32_t)(phase >> 32), quarter = (high + 0x20000000u) & 0xC0000000u;   // nearest quarter turn
  // what is left, in two words (a 64-bit conversion takes several times as long as two): units of 2 pi / 2^32 and / 2^64
  const float x = fmaf((float)(int32_t)(high - quarter), 0x1.921fb6p-30f, (float)(uint32_t)phase * 0x1.921fb6p-62f);
  const float z = x * x;
  const float s = x * fmaf(z, fmaf(z, fmaf(z, fmaf(z, a.sine[4], a.sine[3]), a.sine[2]), a.sine[1]), a.sine[0]);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, a.cosine[4], a.cosine[3]), a.cosine[2]), a.cosine[1]), a.cosine[0]);
  const bool swap = (quarter & 0x40000000u) != 0u;
  const uint32_t cv = __float_as_uint(swap ? s : c) ^ ((quarter + 0x40000000u) & 0x80000000u);
  const uint32_t sv = __float_as_uint(swap ? c : s) ^ (quarter & 0x80000000u);
  float* o = a.out + row * (2 * a.half) + i;
  o[0] = __uint_as_float(cv);
  o[a.half] = __uint_as_float(sv);
}

__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ TableArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();                          // the buffer's readers before this kernel are done
  const int i = (int)threadIdx.x % a.half, r = (int)threadIdx.x / a.half;
  if (r >= a.rows) return;
  const uint64_t w = a.turn[i];
  const int64_t step = (int64_t)gridDim.x * a.rows;
  int64_t row = (int64_t)blockIdx.x * a.rows + r;
  uint64_t phase = (uint64_t)(a.pos0 + row) * w;
  const uint64_t dphase = (uint64_t)step * w;
#pragma unroll 4
  for (; row < a.n; row += step, phase += dphase) write_angle(a, row, i, phase);
}

// ------------------------------------------------------------------ heads
struct HeadArgs {
  const void* q;             // [T, H] heads of D elements: token t, head h at t ldq + h hq
  void* qo;
  int64_t ldq, hq, ldqo, hqo;
  const void* k;             // [T, Hkv] heads, D apart
  void* ko;                  // nullable
  int64_t ldk, ldko;
  const void* v;             // nullable
  int64_t ldv;
  dsa_kv_cache kv;           // kv.k == NULL: none
  const int64_t* slot;
  int H, Hkv, heads;         // heads: of a token in all (queries, keys, values)
  const float* gq;           // nullable together with gk where there is no norm
  const float* gk;
  float eps, inv_d;
  const int32_t* positions;
  const float* cos_sin;
  int64_t max_pos;
  int R, off, D;
  float sign;                // -1: the rotation is taken back
  int64_t T;
  int chunks, q_chunks, k_chunks;   // vector kernel: groups of kHeadsPer heads of a token, of queries, of keys
};

constexpr int kHeadsPer = 4;                       // heads a lane group takes at a time, their loads in flight together

// The pool row of a token, or -1: none (a negative slot) or out of range.
__device__ __forceinline__ int64_t cache_offset(const HeadArgs& a, int64_t t) {
  const int64_t s = a.slot[t];
  if (s < 0) return -1;
  const int64_t rows = a.kv.num_blocks * a.kv.block_size;
  if (s >= rows) {
    raise_error(DSA_DEVERR_INDEX);
    return -1;
  }
  int64_t blk, at;
  if (rows <= 0x7FFFFFFF) {                        // a 64-bit division costs several times as much
    blk = (uint32_t)s / (uint32_t)a.kv.block_size;
    at = (uint32_t)s % (uint32_t)a.kv.block_size;
  } else {
    blk = s / a.kv.block_size;
    at = s % a.kv.block_size;
  }
  return blk * a.kv.block_stride + at * a.kv.row_stride;
}

template <bool F32>
struct Unit;                                       // four neighbouring elements of a head
template <>
struct Unit<false> {
  using Raw = uint2;
  static constexpr int kSize = 2;
  static __device__ __forceinline__ void widen(const Raw& r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x << 16), f[1] = __uint_as_float(r.x & 0xFFFF0000u);
    f[2] = __uint_as_float(r.y << 16), f[3] = __uint_as_float(r.y & 0xFFFF0000u);
  }
};
template <>
struct Unit<true> {
  using Raw = float4;
  static constexpr int kSize = 4;
  static __device__ __forceinline__ void widen(const Raw& r, float (&f)[4]) { f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w; }
};

__device__ __forceinline__ void store4_bf16(void* base, int64_t at, const float (&f)[4]) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]), hi = __floats2bfloat162_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + at) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}
template <bool F32>
__device__ __forceinline__ void store4(void* base, int64_t at, const float (&f)[4]) {
  if constexpr (F32) *reinterpret_cast<float4*>(static_cast<float*>(base) + at) = make_float4(f[0], f[1], f[2], f[3]);
  else store4_bf16(base, at, f);
}

// A group of 2^kLg lanes holds a head, two units of four elements per lane, so that both elements of every pair are in
// one lane: in the half layout unit a of the first half and its partner of the second; interleaved pairs lie within a
// unit.  Both ways a warp's access covers whole neighbouring sectors.  A group takes kHeadsPer heads of one token and one
// kind (query, key, value) at a time: their loads are in flight together, and addresses, cos, sin and the gains are found
// once for them.
template <bool F32, bool kNorm, bool kHalf, int kLg>
__global__ void __launch_bounds__(256) rope_heads_kernel(const __grid_constant__ HeadArgs a) {
  using U = Unit<F32>;
  const int l = (int)threadIdx.x & ((1 << kLg) - 1);
  const int units = a.D >> 2;
  // the lane's units, and whether they turn
  int ua, ub;
  bool ra, rb;
  if constexpr (kHalf) {
    const int rot = a.R >> 3, o = a.off >> 2;      // pairs of units that turn
    if (l < rot) {
      ua = o + l, ub = ua + rot;
      ra = rb = true;
    } else {
      const int p = 2 * (l - rot), skip = a.R >> 2;
      ua = p < o ? p : p + skip;
      ub = p + 1 < o ? p + 1 : p + 1 + skip;
      ra = rb = false;
    }
  } else {
    ua = l, ub = l + (units >> 1);
    ra = 4 * ua >= a.off && 4 * ua < a.off + a.R;
    rb = 4 * ub >= a.off && 4 * ub < a.off + a.R;
  }
  const bool live = 2 * l < units;
  if (!live) ua = ub = 0, ra = rb = false;
  const int da = 4 * ua, db = 4 * ub;
  grid_launch_dependents();
  grid_dependency_wait();

  const uint32_t total = (uint32_t)(a.T * a.chunks);
  const uint32_t step = gridDim.x * (256u >> kLg);
  for (uint32_t c = blockIdx.x * (256u >> kLg) + (threadIdx.x >> kLg); __any_sync(0xFFFFFFFFu, c < total); c += step) {
    const bool on = live && c < total;
    const int64_t t = c / (uint32_t)a.chunks;
    const int j = (int)(c - (uint32_t)t * (uint32_t)a.chunks);
    const int kind = j < a.q_chunks ? 0 : j < a.q_chunks + a.k_chunks ? 1 : 2;
    const int h0 = (kind == 0 ? j : kind == 1 ? j - a.q_chunks : j - a.q_chunks - a.k_chunks) * kHeadsPer;
    const int n = on ? min(kHeadsPer, (kind == 0 ? a.H : a.Hkv) - h0) : 0;
    const int64_t hop = kind == 0 ? a.hq : a.D;    // from head to head
    const int64_t from = (kind == 0 ? t * a.ldq : kind == 1 ? t * a.ldk : t * a.ldv) + h0 * hop;
    const char* src = static_cast<const char*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + from * U::kSize;
    typename U::Raw xa[kHeadsPer], xb[kHeadsPer];
#pragma unroll
    for (int u = 0; u < kHeadsPer; ++u) {
      xa[u] = typename U::Raw{};
      xb[u] = typename U::Raw{};
      if (u < n) {
        xa[u] = *reinterpret_cast<const typename U::Raw*>(src + (u * hop + da) * U::kSize);
        xb[u] = *reinterpret_cast<const typename U::Raw*>(src + (u * hop + db) * U::kSize);
      }
    }
    // cos and sin of the lane's pairs: pair j of unit a (of both units in the half layout) at cs[j], sn[j]
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    bool known = true;
    if (on && (ra || rb) && kind < 2) {
      const int64_t pos = a.positions[t];
      known = pos >= 0 && pos < a.max_pos;
      if (known) {
        const float* row = a.cos_sin + pos * a.R;
        if constexpr (kHalf) {
          const float4 c4 = *reinterpret_cast<const float4*>(row + 4 * l);
          const float4 s4 = *reinterpret_cast<const float4*>(row + (a.R >> 1) + 4 * l);
          cs[0] = c4.x, cs[1] = c4.y, cs[2] = c4.z, cs[3] = c4.w;
          sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
        } else {
          if (ra) {
            const float2 c2 = *reinterpret_cast<const float2*>(row + ((da - a.off) >> 1));
            const float2 s2 = *reinterpret_cast<const float2*>(row + (a.R >> 1) + ((da - a.off) >> 1));
            cs[0] = c2.x, cs[1] = c2.y, sn[0] = s2.x, sn[1] = s2.y;
          }
          if (rb) {
            const float2 c2 = *reinterpret_cast<const float2*>(row + ((db - a.off) >> 1));
            const float2 s2 = *reinterpret_cast<const float2*>(row + (a.R >> 1) + ((db - a.off) >> 1));
            cs[2] = c2.x, cs[3] = c2.y, sn[2] = s2.x, sn[3] = s2.y;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sn[e] *= a.sign;
      } else {                                     // rotated dims become zeros
        raise_error(DSA_DEVERR_INDEX);
      }
    }
    // where the heads go: rows of `type`, rows of the cache, both
    char* dst = nullptr;
    int64_t dst_hop = a.D;
    uint16_t* page = nullptr;
    if (on) {
      if (kind == 0) {
        dst = static_cast<char*>(a.qo) + (t * a.ldqo + h0 * a.hqo) * U::kSize;
        dst_hop = a.hqo;
      } else {
        if (kind == 1 && a.ko != nullptr) dst = static_cast<char*>(a.ko) + (t * a.ldko + (int64_t)h0 * a.D) * U::kSize;
        if (a.kv.k != nullptr) {
          const int64_t at = cache_offset(a, t);
          if (at >= 0) page = static_cast<uint16_t*>(kind == 1 ? a.kv.k : a.kv.v) + at + h0 * a.kv.head_stride;
        }
      }
    }
    // Behind a norm every element is r (x p + partner q): p and q hold the gains and the rotation, and are found once.
    // (For dims that do not turn, q and what it multiplies are zero, whatever the other gain is.)
    float pa[4], pb[4], qa[4], qb[4];
    if constexpr (kNorm) {
      float ga[4] = {1.f, 1.f, 1.f, 1.f}, gb[4] = {1.f, 1.f, 1.f, 1.f};
      if (on && kind < 2) {
        const float4 u4 = *reinterpret_cast<const float4*>((kind == 0 ? a.gq : a.gk) + da);
        const float4 v4 = *reinterpret_cast<const float4*>((kind == 0 ? a.gq : a.gk) + db);
        ga[0] = u4.x, ga[1] = u4.y, ga[2] = u4.z, ga[3] = u4.w;
        gb[0] = v4.x, gb[1] = v4.y, gb[2] = v4.z, gb[3] = v4.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int other = kHalf ? e : e ^ 1;
        const float c0 = kHalf ? cs[e] : cs[e >> 1], s0 = kHalf ? sn[e] : sn[e >> 1];
        const float c1 = kHalf ? cs[e] : cs[2 + (e >> 1)], s1 = kHalf ? sn[e] : sn[2 + (e >> 1)];
        pa[e] = ga[e] * c0;
        pb[e] = gb[e] * c1;
        if constexpr (kHalf) {
          qa[e] = ra ? -gb[other] * s0 : 0.f;
          qb[e] = rb ? ga[other] * s1 : 0.f;
        } else {
          qa[e] = ra ? (e & 1 ? ga[other] : -ga[other]) * s0 : 0.f;
          qb[e] = rb ? (e & 1 ? gb[other] : -gb[other]) * s1 : 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kHeadsPer; ++u) {
      float f[4], g[4];
      U::widen(xa[u], f);
      U::widen(xb[u], g);
      if constexpr (kNorm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fmaf(f[e], f[e], fmaf(g[e], g[e], ss));
#pragma unroll
        for (int o = 1 << kLg >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        if (kind < 2) {
          const float r = rsqrtf(fmaf(ss, a.inv_d, a.eps));
          float x[4], y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = ra ? f[e] : 0.f;
            y[e] = rb ? g[e] : 0.f;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[e] = r * fmaf(kHalf ? y[e] : x[e ^ 1], qa[e], f[e] * pa[e]);
            g[e] = r * fmaf(kHalf ? x[e] : y[e ^ 1], qb[e], g[e] * pb[e]);
          }
        }
      } else if constexpr (kHalf) {
        if (ra && kind < 2) {                      // (values: also a turn by cos 1, sin 0 would spread an infinity)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x0 = f[e], x1 = g[e];
            f[e] = x0 * cs[e] - x1 * sn[e];
            g[e] = x0 * sn[e] + x1 * cs[e];
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (ra && kind < 2) {
            const float x0 = f[2 * k], x1 = f[2 * k + 1];
            f[2 * k] = x0 * cs[k] - x1 * sn[k];
            f[2 * k + 1] = x0 * sn[k] + x1 * cs[k];
          }
          if (rb && kind < 2) {
            const float x0 = g[2 * k], x1 = g[2 * k + 1];
            g[2 * k] = x0 * cs[2 + k] - x1 * sn[2 + k];
            g[2 * k + 1] = x0 * sn[2 + k] + x1 * cs[2 + k];
          }
        }
      }
      if (!known) {                                // zeros, whatever the head holds
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (ra) f[e] = 0.f;
          if (rb) g[e] = 0.f;
        }
      }
      if (u >= n) continue;
      if (dst != nullptr) {
        store4<F32>(dst, u * dst_hop + da, f);
        store4<F32>(dst, u * dst_hop + db, g);
      }
      if (page != nullptr) {
        store4_bf16(page, u * a.kv.head_stride + da, f);
        store4_bf16(page, u * a.kv.head_stride + db, g);
      }
    }
  }
}

// Heads at any alignment, of any size up to 256 and with any part that turns: a warp per head, its values in shared
// memory between the norm and the rotation (a pair's elements lie in different lanes).  For what units do not fit; far from
// the copy rate with its accesses of single elements: rotation of 8192 x 64 x 128 at an odd offset 364 us in bf16 and 288 in
// fp32 (floors 40 and 79), 8192 tokens of 64 + 2 x 8 heads with the norm 544 and 440 (50 and 94).
template <bool F32>
__global__ void __launch_bounds__(256) rope_heads_any_kernel(const __grid_constant__ HeadArgs a, bool norm, bool halves) {
  __shared__ float row_s[8][256];
  float* x = row_s[threadIdx.x >> 5];
  const int lane = (int)threadIdx.x & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  const auto load = [&](const void* p, int64_t i) -> float {
    if constexpr (F32) return static_cast<const float*>(p)[i];
    else return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  };
  const auto store = [&](void* p, int64_t i, float f) {
    if constexpr (F32) static_cast<float*>(p)[i] = f;
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f);
  };
  const int64_t total = a.T * a.heads;
  for (int64_t c = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); c < total; c += (int64_t)gridDim.x * 8) {
    const int64_t t = c / a.heads;
    const int h = (int)(c - t * a.heads);
    const void* p = h < a.H ? a.q : h < a.H + a.Hkv ? a.k : a.v;
    const int64_t in = h < a.H ? t * a.ldq + h * a.hq
                     : h < a.H + a.Hkv ? t * a.ldk + (int64_t)(h - a.H) * a.D : t * a.ldv + (int64_t)(h - a.H - a.Hkv) * a.D;
    const bool turns = h < a.H + a.Hkv;
    float f[8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = lane + 32 * i;
      f[i] = d < a.D ? load(p, in + d) : 0.f;
      ss = fmaf(f[i], f[i], ss);
    }
    float r = 1.f;
    const float* g = h < a.H ? a.gq : a.gk;
    if (norm && turns) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      r = rsqrtf(fmaf(ss, a.inv_d, a.eps));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = lane + 32 * i;
      if (d < a.D) x[d] = norm && turns ? f[i] * (r * g[d]) : f[i];
    }
    __syncwarp();
    const int64_t pos = turns && a.R > 0 ? a.positions[t] : 0;
    const bool known = pos >= 0 && pos < a.max_pos;
    if (turns && a.R > 0 && !known && lane == 0) raise_error(DSA_DEVERR_INDEX);
    int64_t at = -1;
    if (h >= a.H && a.kv.k != nullptr) at = cache_offset(a, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = lane + 32 * i, e = d - a.off;
      if (d >= a.D) continue;
      float y = x[d];
      if (turns && e >= 0 && e < a.R) {
        const int hr = a.R >> 1;
        const int pair = halves ? (e < hr ? e : e - hr) : e >> 1;
        const bool second = halves ? e >= hr : (e & 1) != 0;
        const int apart = halves ? hr : 1, partner = second ? d - apart : d + apart;
        if (known) {
          const float cv = a.cos_sin[pos * a.R + pair], sv = a.sign * a.cos_sin[pos * a.R + hr + pair];
          y = second ? x[partner] * sv + y * cv : y * cv - x[partner] * sv;
        } else {
          y = 0.f;
        }
      }
      if (h < a.H) {
        store(a.qo, t * a.ldqo + h * a.hqo + d, y);
      } else if (turns) {
        if (a.ko != nullptr) store(a.ko, t * a.ldko + (int64_t)(h - a.H) * a.D + d, y);
        if (at >= 0) static_cast<__nv_bfloat16*>(a.kv.k)[at + (h - a.H) * a.kv.head_stride + d] = __float2bfloat16_rn(y);
      } else if (at >= 0) {
        static_cast<__nv_bfloat16*>(a.kv.v)[at + (h - a.H - a.Hkv) * a.kv.head_stride + d] = __float2bfloat16_rn(y);
      }
    }
    __syncwarp();                                  // the row is read before the next one overwrites it
  }
}

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), unsigned grid, unsigned block, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <bool F32, bool kNorm, bool kHalf>
cudaError_t launch_vector(const HeadArgs& a, int num_sms, cudaStream_t stream) {
  int lg = 0;
  while ((8 << lg) < a.D) ++lg;
  const int64_t per = 256 >> lg;
  const int64_t blocks = (a.T * a.chunks + per - 1) / per, most = (int64_t)num_sms * 8;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  switch (lg) {
    case 0: return launch_pdl(rope_heads_kernel<F32, kNorm, kHalf, 0>, grid, 256u, stream, a);
    case 1: return launch_pdl(rope_heads_kernel<F32, kNorm, kHalf, 1>, grid, 256u, stream, a);
    case 2: return launch_pdl(rope_heads_kernel<F32, kNorm, kHalf, 2>, grid, 256u, stream, a);
    case 3: return launch_pdl(rope_heads_kernel<F32, kNorm, kHalf, 3>, grid, 256u, stream, a);
    case 4: return launch_pdl(rope_heads_kernel<F32, kNorm, kHalf, 4>, grid, 256u, stream, a);
    default: return launch_pdl(rope_heads_kernel<F32, kNorm, kHalf, 5>, grid, 256u, stream, a);
  }
}

// The vector kernel: whole units of four elements, pairs within a lane, 8-byte (fp32: 16-byte) accesses.
bool units_fit(const HeadArgs& a, bool f32, bool halves) {
  const uintptr_t al = f32 ? 16 : 8;
  const auto ok = [&](const void* p, int64_t ld) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) % al == 0 && ld % 4 == 0); };
  if (a.D % 8 != 0 || a.off % 4 != 0 || a.R % (halves ? 8 : 4) != 0) return false;
  if (reinterpret_cast<uintptr_t>(a.cos_sin) % 16 != 0 || reinterpret_cast<uintptr_t>(a.gq) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(a.gk) % 16 != 0)
    return false;
  if (a.H > 0 && (!ok(a.q, a.ldq) || !ok(a.qo, a.ldqo) || a.hq % 4 != 0 || a.hqo % 4 != 0)) return false;
  if (a.Hkv > 0 && (!ok(a.k, a.ldk) || !ok(a.ko, a.ldko) || !ok(a.v, a.ldv))) return false;
  if (a.kv.k != nullptr && (reinterpret_cast<uintptr_t>(a.kv.k) % 8 != 0 || reinterpret_cast<uintptr_t>(a.kv.v) % 8 != 0 ||
                            a.kv.block_stride % 4 != 0 || a.kv.row_stride % 4 != 0 || a.kv.head_stride % 4 != 0))
    return false;
  return a.T * a.chunks <= 0x7FFFFFFF;
}

cudaError_t launch_heads(HeadArgs a, bool f32, bool norm, bool halves, int num_sms, cudaStream_t stream) {
  a.heads = a.H + a.Hkv + (a.v != nullptr ? a.Hkv : 0);
  a.q_chunks = (a.H + kHeadsPer - 1) / kHeadsPer;
  a.k_chunks = (a.Hkv + kHeadsPer - 1) / kHeadsPer;
  a.chunks = a.q_chunks + a.k_chunks * (a.v != nullptr ? 2 : 1);
  a.inv_d = 1.f / (float)a.D;
  if (units_fit(a, f32, halves)) {
    if (f32) {
      if (norm) return halves ? launch_vector<true, true, true>(a, num_sms, stream) : launch_vector<true, true, false>(a, num_sms, stream);
      return halves ? launch_vector<true, false, true>(a, num_sms, stream) : launch_vector<true, false, false>(a, num_sms, stream);
    }
    if (norm) return halves ? launch_vector<false, true, true>(a, num_sms, stream) : launch_vector<false, true, false>(a, num_sms, stream);
    return halves ? launch_vector<false, false, true>(a, num_sms, stream) : launch_vector<false, false, false>(a, num_sms, stream);
  }
  const int64_t blocks = (a.T * a.heads + 7) / 8, most = (int64_t)num_sms * 8;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  return f32 ? launch_pdl(rope_heads_any_kernel<true>, grid, 256u, stream, a, norm, halves)
             : launch_pdl(rope_heads_any_kernel<false>, grid, 256u, stream, a, norm, halves);
}

}  // namespace

cudaError_t launch_rope_table(const dsa_rope_params& p, int R, int64_t pos0, int64_t n, float* out, int num_sms,
                              cudaStream_t stream) {
  // in more than 64 bits: a frequency's last bit counts p times at position p
  TableArgs a{};
  using wide = long double;
  const wide two_pi = 6.283185307179586476925286766559005768L, base = p.base, factor = p.factor;
  // YaRN ("NTK by parts", Peng et al. 2023): pairs that turn beta_fast times or more within the trained context keep
  // their frequency, those that turn beta_slow times or less are slowed by the factor, between them it is blended
  wide lo = 0, hi = 0;
  if (p.scaling == DSA_ROPE_YARN) {
    const auto pair = [&](double turns) {
      return R * std::log((double)(p.original_max_pos / (two_pi * turns))) / (2.0 * std::log(p.base));
    };
    lo = std::fmax(std::floor(pair(p.beta_fast)), 0.0);
    hi = std::fmin(std::ceil(pair(p.beta_slow)), (double)R - 1.0);
  }
  // the powers one from the other: half a microsecond each by pow on a host whose long double is software, and a
  // product's rounding, 2^-64 or less each, is nothing next to the angle's 2^-22 even at position 2^31
  const wide ratio = std::pow(base, (wide)-2 / R), slower = 1 / factor - 1, to_turns = std::ldexp(1 / two_pi, 64);
  const wide span = hi - lo > (wide)0.001 ? hi - lo : (wide)0.001;
  wide power = 1;
  for (int i = 0; i < R / 2; ++i, power *= ratio) {
    wide f = power * to_turns;
    if (p.scaling == DSA_ROPE_LINEAR) f /= factor;
    if (p.scaling == DSA_ROPE_YARN && i > lo) f += f * slower * (i >= hi && i - lo >= span ? (wide)1 : (i - lo) / span);
    a.turn[i] = (uint64_t)f;                                  // base > 1: less than a turn
  }
  a.pos0 = pos0, a.n = n, a.half = R / 2, a.out = out;
  double odd = p.amplitude, even = p.amplitude;
  for (int k = 0; k < 5; odd /= -(2.0 * k + 2.0) * (2.0 * k + 3.0), even /= -(2.0 * k + 1.0) * (2.0 * k + 2.0), ++k) {
    a.sine[k] = (float)odd;                                   // (-1)^k / (2k + 1)!
    a.cosine[k] = (float)even;                                // (-1)^k / (2k)!
  }
  a.rows = 256 / a.half;
  const int64_t blocks = (n + a.rows - 1) / a.rows, most = (int64_t)num_sms * 8;
  return launch_pdl(rope_table_kernel, (unsigned)(blocks < most ? blocks : most), 256u, stream, a);
}

cudaError_t launch_rope(const void* x, int64_t ldx, int64_t hx, const int32_t* positions, const float* cos_sin,
                        int64_t max_pos, int R, int off, bool halves, bool inverse, int64_t T, int H, int D, bool f32,
                        void* y, int64_t ldy, int64_t hy, int num_sms, cudaStream_t stream) {
  HeadArgs a{};
  if (x == y) {                                    // in place: what does not turn stays where it is
    const int64_t skip = (int64_t)off * (f32 ? 4 : 2);
    x = y = static_cast<char*>(y) + skip;
    D = R, off = 0;
  }
  a.q = x, a.qo = y, a.ldq = ldx, a.hq = hx, a.ldqo = ldy, a.hqo = hy;
  a.positions = positions, a.cos_sin = cos_sin, a.max_pos = max_pos, a.R = R, a.off = off, a.D = D;
  a.sign = inverse ? -1.f : 1.f;
  a.T = T, a.H = H;
  return launch_heads(a, f32, false, halves, num_sms, stream);
}

cudaError_t launch_qk_norm_rope(const void* q, int64_t ldq, int H, const void* k, int64_t ldk, int Hkv, const void* v,
                                int64_t ldv, int64_t T, int D, bool f32, const float* gamma_q, const float* gamma_k,
                                float eps, const int32_t* positions, const float* cos_sin, int64_t max_pos, int R, int off,
                                bool halves, void* q_out, int64_t ldqo, void* k_out, int64_t ldko, const dsa_kv_cache& kv,
                                const int64_t* slot, int num_sms, cudaStream_t stream) {
  HeadArgs a{};
  a.q = q, a.qo = q_out, a.ldq = ldq, a.ldqo = ldqo, a.hq = a.hqo = D;
  a.k = k, a.ko = k_out, a.ldk = ldk, a.ldko = ldko;
  a.v = v, a.ldv = ldv;
  a.kv = kv, a.slot = slot;
  a.positions = positions, a.cos_sin = cos_sin, a.max_pos = max_pos, a.R = R, a.off = off, a.D = D;
  a.gq = gamma_q, a.gk = gamma_k, a.eps = eps;
  a.sign = 1.f;
  a.T = T, a.H = H, a.Hkv = Hkv;
  return launch_heads(a, f32, gamma_q != nullptr || gamma_k != nullptr, halves, num_sms, stream);
}

DSA_DEFINE_TU_ERROR_ACCESSORS(rope)

}  // namespace dsa
