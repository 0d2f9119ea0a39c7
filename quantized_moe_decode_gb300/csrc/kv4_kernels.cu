// The 4-bit KV cache: rotary positions and the append, attention over the
// entries, and the eviction of the entries that attention uses least.
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>

#include "kv4_common.cuh"
#include "launch.h"

namespace uocr {

// ------------------------------------------------------------------ append
// cos and sin of a in double: a is reduced by the nearest multiple of pi/2 in
// two steps and the remainder, at most pi/4, goes through the Taylor series up
// to r^16 / 16! (truncation below 1e-14), so the rounded fp32 results are the
// nearest ones but for about one argument in 1e6.
__device__ __forceinline__ void sincos_taylor(double a, double& sn, double& cs) {
  const double n = rint(a * 0.63661977236758134308);
  double r = fma(-n, 1.57079632679489655800, a);
  r = fma(-n, 6.12323399573676603587e-17, r);
  const double z = r * r;
  double s = -1.0 / 1307674368000.0, c = 1.0 / 20922789888000.0;
  s = fma(s, z, 1.0 / 6227020800.0);
  c = fma(c, z, -1.0 / 87178291200.0);
  s = fma(s, z, -1.0 / 39916800.0);
  c = fma(c, z, 1.0 / 479001600.0);
  s = fma(s, z, 1.0 / 362880.0);
  c = fma(c, z, -1.0 / 3628800.0);
  s = fma(s, z, -1.0 / 5040.0);
  c = fma(c, z, 1.0 / 40320.0);
  s = fma(s, z, 1.0 / 120.0);
  c = fma(c, z, -1.0 / 720.0);
  s = fma(s, z, -1.0 / 6.0);
  c = fma(c, z, 1.0 / 24.0);
  s = fma(s * z, r, r);
  c = fma(c, z, -0.5);
  c = fma(c, z, 1.0);
  const int k = (int)((long long)n & 3);
  const double u = (k & 1) ? c : s, w = (k & 1) ? s : c;
  sn = (k & 2) ? -u : u;
  cs = (k == 1 || k == 2) ? -w : w;
}

// cos and sin of b inv_j (first table) and 256 b inv_j (second), b < 256: what a
// chunk's positions are composed from.  The product's rounding error e enters
// as cos(x + e) = cos x - e sin x.
__global__ void k_kv4_turns(const double* inv_freq, double2* turns, int pairs) {
  const double f = inv_freq[threadIdx.x], b = (double)(blockIdx.x & 255) * (blockIdx.x >> 8 ? 256.0 : 1.0);
  const double x = b * f, e = fma(b, f, -x);
  double sn, cs;
  sincos_taylor(x, sn, cs);
  turns[(size_t)blockIdx.x * pairs + threadIdx.x] = make_double2(fma(-e, sn, cs), fma(e, cs, sn));
}

cudaError_t launch_kv4_turns(const double* inv_freq, double2* turns, int pairs, cudaStream_t st) {
  k_kv4_turns<<<512, pairs, 0, st>>>(inv_freq, turns, pairs);
  return cudaGetLastError();
}

// Eight neighbouring elements in fp32.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* p, long long at, float (&x)[8]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = load_elem(p, DT, at + j);
  } else if constexpr (DT == 0) {
    const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
    const float4 u = __ldg(q), v = __ldg(q + 1);
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
  } else {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned short*>(p) + at));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == 1) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
      } else {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
}

// Place of pair j's (cos, sin) in shared memory: lanes that take pairs 8 apart
// read neighbouring entries.
__device__ __forceinline__ int turn_at(int j) { return (j & 7) * 17 + (j >> 3); }

// Dimensions d .. d+7 of a vector at `base`, rotated: (x, y) -> (x c - y s,
// y c + x s), the products and the sum each rounded to fp32.
template <int DT, bool VEC>
__device__ __forceinline__ void load8_rotated(const void* p, long long base, int d, const Kv4AppendArgs& a,
                                              const float2* cs, float (&x)[8]) {
  load8<DT, VEC>(p, base + d, x);
  const int rd = a.rope_dims, half = rd >> 1;
  if (d >= rd) return;
  if (a.rope_layout == 1) {
#pragma unroll
    for (int j = 0; j < 8; j += 2)
      if (d + j < rd) {
        const float2 r = cs[turn_at((d + j) >> 1)];
        const float u = x[j], v = x[j + 1];
        x[j] = __fsub_rn(__fmul_rn(u, r.x), __fmul_rn(v, r.y));
        x[j + 1] = __fadd_rn(__fmul_rn(v, r.x), __fmul_rn(u, r.y));
      }
    return;
  }
  if ((half & 7) == 0) {  // the partners are eight neighbours too
    const bool lo = d < half;
    const int o = lo ? d + half : d - half, c = lo ? d : d - half;
    float y[8];
    load8<DT, VEC>(p, base + o, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 r = cs[turn_at(c + j)];
      const float u = __fmul_rn(x[j], r.x), v = __fmul_rn(y[j], r.y);
      x[j] = lo ? __fsub_rn(u, v) : __fadd_rn(u, v);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = d + j;
    if (i >= rd) break;
    const bool lo = i < half;
    const float2 r = cs[turn_at(lo ? i : i - half)];
    const float u = __fmul_rn(x[j], r.x), v = __fmul_rn(load_elem(p, DT, base + (lo ? i + half : i - half)), r.y);
    x[j] = lo ? __fsub_rn(u, v) : __fadd_rn(u, v);
  }
}

// One CTA per token; a thread takes eight dimensions of a key, value or query
// vector, four neighbouring lanes a group of 32.  What it cannot do without is
// reading the projections once and writing queries and entries; the rest is
// arithmetic per element (rotation, two divisions' worth of quantising), so the
// loads are 16 bytes wide where the addresses allow (VEC).  Double precision
// runs at 1/64 of the fp32 rate here: a chunk takes its angles from the
// context's two tables with four operations per pair instead of some forty.
template <int DT, bool VEC>
__global__ void __launch_bounds__(1024) k_kv4_append(const Kv4AppendArgs a) {
  __shared__ float2 s_cs[8 * 17];
  pdl_launch_dependents();
  pdl_wait();
  const int t = blockIdx.x, D = a.D;
  int p = a.pos ? a.pos[t] : a.pos0 + t;
  const int row = a.kv_row0 + t * a.kv_rstep;
  bool write = true;
  int slot = p;
  if (!a.slots) {
    const int2 hole = a.hole[row];
    if (p < 0 || (hole.y > hole.x && p < hole.y)) {
      // an evicted prefix has no slot for its positions; a negative one takes position 0
      if (threadIdx.x == 0) atomicOr(a.status, kStatusPosition);
      write = !(hole.y > hole.x);
      p = max(p, 0);
    }
    slot = kv_slot(p, a.P, a.R);
  }
  if (a.rotate) {
    const int pairs = a.rope_dims >> 1;
    for (int j = threadIdx.x; j < pairs; j += blockDim.x) {
      double sn, cs;
      if (!a.pos && p < 65536) {
        const double2 u = a.turns[(size_t)(p & 255) * (D >> 1) + j], v = a.turns[(size_t)(256 + (p >> 8)) * (D >> 1) + j];
        cs = fma(u.x, v.x, -(u.y * v.y));
        sn = fma(u.y, v.x, u.x * v.y);
      } else {
        sincos_taylor((double)p * a.inv_freq[j], sn, cs);
      }
      s_cs[turn_at(j)] = make_float2((float)(a.amp * cs), (float)(a.amp * sn));
    }
    __syncthreads();
  }
  const int wpv = D >> 3, lw = 31 - __clz(wpv);  // words per vector, a power of two
  uint8_t* row4 = a.kv4 + (size_t)row * 2 * a.nh * a.tiles * kv4_tile_bytes(D);
  const int tile = slot >> 4, s = slot & 15;
  const int kv_items = 2 * a.nh << lw, total = kv_items + (a.q_heads << lw);  // multiples of 4
  for (int i0 = 0; i0 < total; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    const int vec = i >> lw, w = i & (wpv - 1);
    float x[8];
    if (i >= kv_items) {
      if (i < total) {
        const int h = vec - 2 * a.nh;
        load8_rotated<DT, VEC>(a.q, t * a.ldq + (long long)h * D, 8 * w, a, s_cs, x);
        float4* o = reinterpret_cast<float4*>(a.q_out + ((size_t)t * a.q_heads + h) * D + 8 * w);
        if (VEC) {
          o[0] = make_float4(x[0], x[1], x[2], x[3]);
          o[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) reinterpret_cast<float*>(o)[j] = x[j];
        }
      }
    }
    const bool in = i < kv_items;
    if (!__any_sync(0xffffffffu, in)) continue;
    const int kv = vec >= a.nh, head = kv ? vec - a.nh : vec;
    float mn = INFINITY, mx = -INFINITY;
    bool ok = true;
    if (in) {
      if (kv)
        load8<DT, VEC>(a.v, t * a.ldv + head * a.lhk + 8 * w, x);
      else if (a.rotate)
        load8_rotated<DT, VEC>(a.k, t * a.ldk + head * a.lhk, 8 * w, a, s_cs, x);
      else
        load8<DT, VEC>(a.k, t * a.ldk + head * a.lhk + 8 * w, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mn = fminf(mn, x[j]);
        mx = fmaxf(mx, x[j]);
        ok = ok && fabsf(x[j]) <= 65504.f;
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      ok = __shfl_xor_sync(0xffffffffu, (int)ok, o) && ok;
    }
    if (!in) continue;
    __half sc, lo;
    kv4_params(mn, mx, ok, sc, lo);
    const float sf = __half2float(sc), mf = __half2float(lo);
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = kv4_code(x[j], sf, mf);
    __half* val = kv ? a.v_val : a.k_val;
    if (val) {
      val += ((size_t)t * a.nh + head) * D + 8 * w;
      uint32_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2 h = __halves2half2(kv4_value(c[2 * j], sc, lo), kv4_value(c[2 * j + 1], sc, lo));
        v[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if (VEC) {
        *reinterpret_cast<uint4*>(val) = make_uint4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) val[j] = __ushort_as_half((unsigned short)(v[j >> 1] >> (16 * (j & 1))));
      }
    }
    if (!write) continue;
    uint8_t* tp = row4 + ((size_t)(kv * a.nh + head) * a.tiles + tile) * kv4_tile_bytes(D);
    const int grp = w >> 2;
    if (!kv) {
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) word |= c[j] << (4 * ((j >> 1) + 4 * (j & 1)));
      *reinterpret_cast<uint32_t*>(tp + kv4_k_word(D, s, w)) = word;
      if ((w & 3) == 0) {
        *reinterpret_cast<__half2*>(tp + kv4_k_param(D, s, grp)) = __halves2half2(sc, lo);
        if (a.wts && w == 0) a.wts[((size_t)row * a.nh + head) * a.tiles * kKv4Slots + slot] = 0.f;
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<uint16_t*>(tp + kv4_v_quad(D, s, 2 * w + h)) =
            (uint16_t)(c[4 * h] | (c[4 * h + 1] << 4) | (c[4 * h + 2] << 8) | (c[4 * h + 3] << 12));
      if ((w & 3) == 0) {
        *reinterpret_cast<__half*>(tp + kv4_v_param(D, s, grp, 0)) = sc;
        *reinterpret_cast<__half*>(tp + kv4_v_param(D, s, grp, 1)) = lo;
      }
    }
  }
}

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int tokens, cudaStream_t st, bool pdl) {
  if (tokens <= 0) return cudaSuccess;
  const long long e = a.dtype == 0 ? 4 : 2;
  auto wide = [&](const void* p, long long ld) { return ((uintptr_t)p | (uintptr_t)(ld * e)) % 16 == 0; };
  const bool vec = wide(a.q, a.ldq) && wide(a.k, a.ldk) && wide(a.v, a.ldv) && a.lhk * e % 16 == 0 &&
                   ((uintptr_t)a.q_out | (uintptr_t)a.k_val | (uintptr_t)a.v_val) % 16 == 0;
  // few tokens: one round of threads over the vectors, so that a step waits for one load
  const int items = (2 * a.nh + a.q_heads) * (a.D / 8);
  const int threads = tokens >= a.n_sm || items <= 256 ? 256 : items <= 512 ? 512 : 1024;
#define UOCR_APPEND(DT_)                                                                                       \
  return vec ? launch_kernel(k_kv4_append<DT_, true>, dim3(tokens), dim3(threads), 0, st, pdl, a)              \
             : launch_kernel(k_kv4_append<DT_, false>, dim3(tokens), dim3(threads), 0, st, pdl, a);
  switch (a.dtype) {
    case 0: UOCR_APPEND(0)
    case 1: UOCR_APPEND(1)
    case 2: UOCR_APPEND(2)
  }
#undef UOCR_APPEND
  return cudaErrorInvalidValue;
}

__global__ void k_kv4_zero(const Kv4AppendArgs a, int row, int slot0) {
  const int slot = slot0 + blockIdx.x, head = blockIdx.y, s = slot & 15, D = a.D;
  uint8_t* kp = a.kv4 + ((size_t)(row * 2 * a.nh + head) * a.tiles + (slot >> 4)) * kv4_tile_bytes(D);
  uint8_t* vp = kp + (size_t)a.nh * a.tiles * kv4_tile_bytes(D);
  for (int w = threadIdx.x; w < D / 4; w += blockDim.x) {
    if (w < D / 8) *reinterpret_cast<uint32_t*>(kp + kv4_k_word(D, s, w)) = 0u;
    *reinterpret_cast<uint16_t*>(vp + kv4_v_quad(D, s, w)) = 0;
    if (w < D / 32) *reinterpret_cast<uint32_t*>(kp + kv4_k_param(D, s, w)) = 0u;
    if (w < D / 16) *reinterpret_cast<uint16_t*>(vp + kv4_v_param(D, s, w >> 1, w & 1)) = 0;
  }
  if (a.wts && threadIdx.x == 0) a.wts[((size_t)row * a.nh + head) * a.tiles * kKv4Slots + slot] = 0.f;
}

cudaError_t launch_kv4_zero(const Kv4AppendArgs& a, int row, int slot0, int n, cudaStream_t st) {
  if (n <= 0) return cudaSuccess;
  k_kv4_zero<<<dim3(n, a.nh), 32, 0, st>>>(a, row, slot0);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ entries
// dimensions 8w .. 8w+7 of a key entry, dimensions 4i .. 4i+3 of a value entry
__device__ __forceinline__ void key_values(const uint8_t* tp, int D, int s, int w, __half (&x)[8]) {
  const uint32_t word = *reinterpret_cast<const uint32_t*>(tp + kv4_k_word(D, s, w));
  const __half2 p = *reinterpret_cast<const __half2*>(tp + kv4_k_param(D, s, w >> 2));
#pragma unroll
  for (int j = 0; j < 8; ++j)
    x[j] = kv4_value((word >> (4 * ((j >> 1) + 4 * (j & 1)))) & 15u, __low2half(p), __high2half(p));
}
__device__ __forceinline__ void value_values(const uint8_t* tp, int D, int s, int i, __half (&x)[4]) {
  const uint32_t q = *reinterpret_cast<const uint16_t*>(tp + kv4_v_quad(D, s, i));
  const __half sc = *reinterpret_cast<const __half*>(tp + kv4_v_param(D, s, i >> 3, 0));
  const __half lo = *reinterpret_cast<const __half*>(tp + kv4_v_param(D, s, i >> 3, 1));
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = kv4_value((q >> (4 * j)) & 15u, sc, lo);
}

// One warp per (slot, K|V, head): entries to and from the callers' layout.
__global__ void k_kv4_io(const Kv4IoArgs a) {
  const int i = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= a.n) return;
  const int head = blockIdx.y, kv = blockIdx.z, D = a.D, NG = D / kKv4Group;
  const int slot = a.slot0 + i, s = slot & 15;
  uint8_t* tp = a.kv4 + ((size_t)(kv * a.nh + head) * a.tiles + (slot >> 4)) * kv4_tile_bytes(D);
  const size_t vec = (size_t)head * a.n + i;
  if (a.val[kv]) {
    for (int w = lane; w < D / 4; w += 32) {
      __half* out = a.val[kv] + vec * D + 4 * w;
      if (kv) {
        __half x[4];
        value_values(tp, D, s, w, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = x[j];
      } else {
        __half x[8];
        key_values(tp, D, s, w >> 1, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = (w & 1) ? x[4 + j] : x[j];
      }
    }
    return;
  }
  uint8_t* codes = a.codes[kv] + vec * D;
  for (int w = lane; w < D / 8; w += 32) {
    if (kv) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint16_t* q = reinterpret_cast<uint16_t*>(tp + kv4_v_quad(D, s, 2 * w + h));
        uint32_t u = 0;
        if (a.put) {
#pragma unroll
          for (int j = 0; j < 4; ++j) u |= (uint32_t)(codes[8 * w + 4 * h + j] & 15) << (4 * j);
          *q = (uint16_t)u;
        } else {
          u = *q;
#pragma unroll
          for (int j = 0; j < 4; ++j) codes[8 * w + 4 * h + j] = (u >> (4 * j)) & 15;
        }
      }
    } else {
      uint32_t* q = reinterpret_cast<uint32_t*>(tp + kv4_k_word(D, s, w));
      uint32_t u = 0;
      if (a.put) {
#pragma unroll
        for (int j = 0; j < 8; ++j) u |= (uint32_t)(codes[8 * w + j] & 15) << (4 * ((j >> 1) + 4 * (j & 1)));
        *q = u;
      } else {
        u = *q;
#pragma unroll
        for (int j = 0; j < 8; ++j) codes[8 * w + j] = (u >> (4 * ((j >> 1) + 4 * (j & 1)))) & 15;
      }
    }
  }
  for (int g = lane; g < NG; g += 32) {
    __half* sp = kv ? reinterpret_cast<__half*>(tp + kv4_v_param(D, s, g, 0))
                    : reinterpret_cast<__half*>(tp + kv4_k_param(D, s, g));
    __half* mp = kv ? reinterpret_cast<__half*>(tp + kv4_v_param(D, s, g, 1)) : sp + 1;
    if (a.put) {
      *sp = a.scale[kv][vec * NG + g];
      *mp = a.low[kv][vec * NG + g];
    } else {
      a.scale[kv][vec * NG + g] = *sp;
      a.low[kv][vec * NG + g] = *mp;
    }
  }
  if (a.put && a.wts && !kv && lane == 0) a.wts[(size_t)head * a.tiles * kKv4Slots + slot] = 0.f;
}

cudaError_t launch_kv4_io(const Kv4IoArgs& a, cudaStream_t st) {
  if (a.n <= 0) return cudaSuccess;
  k_kv4_io<<<dim3((a.n + 7) / 8, a.nh, 2), 256, 0, st>>>(a);
  return cudaGetLastError();
}

__global__ void k_kv4_weights(const Kv4WeightsArgs a) {
  const int head = blockIdx.y % a.nh, r = blockIdx.y / a.nh, l = blockIdx.z;
  float* w = a.wts + (((size_t)(a.layer0 + l) * a.MR + a.row0 + r) * a.nh + head) * a.tiles * kKv4Slots + a.slot0;
  float* d = a.dense + (((size_t)l * a.rows + r) * a.nh + head) * a.n;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.n; i += gridDim.x * blockDim.x) {
    if (a.put)
      w[i] = d[i];
    else
      d[i] = w[i];
  }
}

cudaError_t launch_kv4_weights(const Kv4WeightsArgs& a, cudaStream_t st) {
  if (a.n <= 0) return cudaSuccess;
  const int gx = (a.n + 1023) / 1024;
  k_kv4_weights<<<dim3(gx < 64 ? gx : 64, a.rows * a.nh, a.layers), 256, 0, st>>>(a);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ attention
// softmax(q k / sqrt D) v over the live slots, split over a cluster of CTAs.
//
// A CTA holds the queries that read one (row, head): the heads that share it,
// or a tile of a chunk's tokens.  A warp takes 16-slot tiles in turn and keeps
// an online softmax per query.  Both products run on the tensor cores with the
// cache as the A operand (m16n8k16): scores = K q with slots as rows, then
// out = V^T p with dimensions as rows.  The cache's layout puts the A fragments
// into a lane's own bytes, so a lane copies them with cp.async into its own
// ring slots (no barrier guards them), turns a word of eight codes into four
// fp16 pairs with three masks and a shift, and applies scale and minimum with
// one fused multiply-add each, which gives the entry's value exactly.
//
// The eight B columns are four queries, each as an fp16 number and the fp16
// remainder of its fp32 value (queries scaled by a power of two to [1, 2)), and
// likewise the four weight vectors: the products then carry about 22 bits at
// no cost, since a decode step would leave the columns empty.  Scores, sums and
// outputs accumulate in fp32.  The running maximum of a query moves only when
// a score exceeds it by 2^8 (weights up to 256 are held), so that almost no tile
// rescales the accumulators.
constexpr int kAttn4Warps = 8;
constexpr int kAttn4Stages = 4;  // tiles of a warp's ring

template <int D>
struct Attn4 {
  static constexpr int NG = D / 32;
  static constexpr int CB = D / 4;                // code bytes of a lane in a K or V tile
  static constexpr int KPB = D == 256 ? 16 : 8;   // its key parameter bytes
  static constexpr int STAGE = 32 * (2 * CB + KPB + 16);
  static constexpr int RING = kAttn4Stages * STAGE;
};

// One exponential; the argument is in units of log2.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t hfma2u(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hsub2u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Four pairs of codes of a word (nibbles 0|4, 1|5, 2|6, 3|7) as fp16 values
// s q + m: the code is or'ed into the mantissa of 1024 (bits 0-3) or 64 (bits
// 4-7), which is subtracted again, exactly.
__device__ __forceinline__ void dequant8(uint32_t w, uint32_t s, uint32_t m, uint32_t (&x)[4]) {
  const uint32_t h = w >> 8;
  x[0] = hfma2u(s, hsub2u(lop_and_or(w, 0x000F000Fu, 0x64006400u), 0x64006400u), m);
  x[1] = hfma2u(s, hsub2u(lop_and_or(w, 0x00F000F0u, 0x54005400u), 0x54005400u), m);
  x[2] = hfma2u(s, hsub2u(lop_and_or(h, 0x000F000Fu, 0x64006400u), 0x64006400u), m);
  x[3] = hfma2u(s, hsub2u(lop_and_or(h, 0x00F000F0u, 0x54005400u), 0x54005400u), m);
}

// The slots a CTA reads, as whole tiles: those of [0, x) and of [y, lim).
struct TileList {
  int ta, tb, count;
  __device__ TileList(int lim, int2 hole) {
    const int x = min(hole.x, lim);
    const bool gap = hole.y > hole.x && lim > hole.x;
    ta = ((gap ? x : lim) + 15) >> 4;
    tb = gap ? max(ta, hole.y >> 4) : ta;
    count = ta + (gap && lim > hole.y ? max(((lim + 15) >> 4) - tb, 0) : 0);
  }
  __device__ int operator()(int j) const { return j < ta ? j : tb + (j - ta); }
};

template <int D, int NT>
__global__ void __launch_bounds__(kAttn4Warps * 32, D * NT <= 128 ? 2 : 1) k_kv4_attn(const Kv4AttnArgs a, int n_queries) {
  using C = Attn4<D>;
  constexpr int NW = kAttn4Warps, ST = kAttn4Stages, NQ = 4 * NT;
  constexpr bool QREG = D * NT <= 256;  // query fragments in registers, else in shared memory
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float s_m[NW][NQ], s_l[NW][NQ];
  __shared__ float s_part[NQ][D + 2];
  __shared__ float s_c[NQ];     // score factor of each query: scale log2(e) 2^e
  __shared__ float2 s_fin[NQ];  // final maximum and 1 / sum
  __shared__ int s_lim[NQ];
  __shared__ uint2 s_q[QREG ? 1 : NT * (D / 16) * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, head = blockIdx.y, G = a.q_heads / a.nh;
  // queries of this CTA: u = token * G + head in the group
  const int u0 = a.kv_rstep ? blockIdx.z * G : blockIdx.z * NQ;
  const int nq = a.kv_rstep ? G : min(NQ, n_queries - u0);
  const int row = a.kv_row0 + (a.kv_rstep ? blockIdx.z : 0);
  auto token = [&](int i) { return (u0 + i) / G; };
  auto q_index = [&](int i) { return (size_t)token(i) * a.q_heads + head * G + (u0 + i) % G; };

  pdl_launch_dependents();
  pdl_wait();  // queries and new entries come from the previous kernels
  const int2 hole = a.hole[row];
  if (threadIdx.x < NQ) {
    int lim = 0;
    if (threadIdx.x < nq) {
      const int tok = token(threadIdx.x);
      int p = a.pos ? a.pos[tok] : a.pos0 + tok;
      if (p < 0 || (hole.y > hole.x && p < hole.y)) {
        atomicOr(a.status, kStatusPosition);
        p = max(p, 0);
      }
      lim = kv_limit(p, a.P, a.R);
    }
    s_lim[threadIdx.x] = lim;
  }
  // queries to fp16 pairs (value, remainder): a warp per query
  float* sq = reinterpret_cast<float*>(smem);  // [NQ][D], before the ring is used
  for (int i = warp; i < NQ; i += NW) {
    float mx = 0.f;
    for (int d = lane; d < D; d += 32) {
      const float x = i < nq ? a.q[q_index(i) * D + d] : 0.f;
      sq[i * D + d] = x;
      mx = fmaxf(mx, fabsf(x));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // 2^-e with e the exponent of the largest magnitude (0 and infinities stay)
    const int e = mx > 0.f && mx < INFINITY ? min(max(ilogbf(mx), -100), 100) : 0;
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    for (int d = lane; d < D; d += 32) sq[i * D + d] *= down;
    if (lane == 0) s_c[i] = a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23);
  }
  __syncthreads();
  uint2 qf[QREG ? NT * (D / 16) : 1];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      // step k covers dimensions 8 (k/2) + 4 (k%2) .. + 3 of every lane's quarter
      const float* s = sq + (4 * nt + (g >> 1)) * D + t * (D / 4) + 4 * k;
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float hi = __half2float(__float2half_rn(s[j]));
        v[j] = (g & 1) ? s[j] - hi : s[j];
      }
      const uint2 f = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
      if constexpr (QREG)
        qf[nt * (D / 16) + k] = f;
      else if (warp == 0)
        s_q[(nt * (D / 16) + k) * 32 + lane] = f;
    }
  int lim_lo = INT_MAX, lim_hi = 0;
  for (int i = 0; i < nq; ++i) {
    lim_lo = min(lim_lo, s_lim[i]);
    lim_hi = max(lim_hi, s_lim[i]);
  }
  int lim_q[NT];
  float cq[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    lim_q[nt] = s_lim[4 * nt + t];
    cq[nt] = s_c[4 * nt + t];
  }
  __syncthreads();  // the ring overwrites sq

  const TileList tiles(lim_hi, hole);
  const int per = (tiles.count + gridDim.x - 1) / gridDim.x;
  const int j0 = split * per, j1 = min(tiles.count, j0 + per);
  const uint8_t* kt = a.kv4 + ((size_t)row * 2 * a.nh + head) * a.tiles * kv4_tile_bytes(D);
  const uint8_t* vt = kt + (size_t)a.nh * a.tiles * kv4_tile_bytes(D);
  unsigned char* ring = smem + warp * C::RING;
  const int kp_off = 8 * D + (D == 256 ? g * 64 + t * 16 : (g * C::NG + t * C::NG / 4) * 8);
  const int vp_off = 8 * D + ((g * D / 256) * 4 + t) * 16;
  auto issue = [&](int j, int stage) {
    if (j < j1) {
      const size_t off = (size_t)tiles(j) * kv4_tile_bytes(D);
      unsigned char* d = ring + stage * C::STAGE;
      if constexpr (D == 32) {
        cp_async8(d + lane * 8, kt + off + lane * 8);
        cp_async8(d + 32 * C::CB + lane * 8, vt + off + lane * 8);
      } else {
#pragma unroll
        for (int p = 0; p < C::CB / 16; ++p) {
          cp_async16(d + p * 512 + lane * 16, kt + off + p * 512 + lane * 16);
          cp_async16(d + 32 * C::CB + p * 512 + lane * 16, vt + off + p * 512 + lane * 16);
        }
      }
      if constexpr (C::KPB == 16)
        cp_async16(d + 64 * C::CB + lane * 16, kt + off + kp_off);
      else
        cp_async8(d + 64 * C::CB + lane * 8, kt + off + kp_off);
      cp_async16(d + 64 * C::CB + 32 * C::KPB + lane * 16, vt + off + vp_off);
    }
    cp_commit();
  };

  float m_ref[NT], l[NT], acc[NT][D / 16][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m_ref[nt] = -INFINITY;
    l[nt] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[nt][i][j] = 0.f;
  }
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) issue(j0 + warp + s * NW, s);

  int stage = 0;
  for (int j = j0 + warp; j < j1; j += NW) {
    cp_wait<ST - 2>();
    const unsigned char* d = ring + stage * C::STAGE;
    issue(j + (ST - 1) * NW, stage == 0 ? ST - 1 : stage - 1);  // the slot that the last tile left
    stage = stage == ST - 1 ? 0 : stage + 1;
    const int slot0 = tiles(j) * 16;
    const bool gap = hole.y > hole.x;
    const bool full = slot0 + 16 <= lim_lo && (!gap || slot0 + 16 <= hole.x || slot0 >= hole.y);

    // ---- scores
    float sc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[nt][i] = 0.f;
    {
      constexpr int W = D / 32;  // words per slot
      uint32_t w[2 * W];
      if constexpr (D == 32) {
        const uint2 u = *reinterpret_cast<const uint2*>(d + lane * 8);
        w[0] = u.x;
        w[1] = u.y;
      } else {
#pragma unroll
        for (int p = 0; p < W / 2; ++p) {
          const uint4 u = lds128(d + p * 512 + lane * 16);
          w[4 * p] = u.x;
          w[4 * p + 1] = u.y;
          w[4 * p + 2] = u.z;
          w[4 * p + 3] = u.w;
        }
      }
      // (s, m) of slots g and g + 8, one or two groups
      uint32_t par[4];
      if constexpr (C::KPB == 16) {
        const uint4 u = lds128(d + 64 * C::CB + lane * 16);
        par[0] = u.x, par[1] = u.y, par[2] = u.z, par[3] = u.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(d + 64 * C::CB + lane * 8);
        par[0] = u.x, par[1] = u.y, par[2] = u.x, par[3] = u.y;
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint32_t p0 = par[i >= 4 ? 2 : 0], p1 = par[i >= 4 ? 3 : 1];
        uint32_t e[4], f[4];
        dequant8(w[i], __byte_perm(p0, 0, 0x1010), __byte_perm(p0, 0, 0x3232), e);
        dequant8(w[W + i], __byte_perm(p1, 0, 0x1010), __byte_perm(p1, 0, 0x3232), f);
        const uint32_t a0[4] = {e[0], f[0], e[1], f[1]}, a1[4] = {e[2], f[2], e[3], f[3]};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint2 b0, b1;
          if constexpr (QREG) {
            b0 = qf[nt * (D / 16) + 2 * i];
            b1 = qf[nt * (D / 16) + 2 * i + 1];
          } else {
            b0 = s_q[(nt * (D / 16) + 2 * i) * 32 + lane];
            b1 = s_q[(nt * (D / 16) + 2 * i + 1) * 32 + lane];
          }
          mma_16816(sc[nt], a0, b0.x, b0.y);
          mma_16816(sc[nt], a1, b1.x, b1.y);
        }
      }
    }
    // ---- softmax: lane (g, t) holds slots g and g + 8 of query t
    float p0[NT], p1[NT];
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      p0[nt] = (sc[nt][0] + sc[nt][1]) * cq[nt];
      p1[nt] = (sc[nt][2] + sc[nt][3]) * cq[nt];
      if (!full) {
        const int s0 = slot0 + g, s1 = s0 + 8;
        if (s0 >= lim_q[nt] || (s0 >= hole.x && s0 < hole.y)) p0[nt] = -INFINITY;
        if (s1 >= lim_q[nt] || (s1 >= hole.x && s1 < hole.y)) p1[nt] = -INFINITY;
      }
      if (a.scores && 4 * nt + t < nq) {
        float* so = a.scores + q_index(4 * nt + t) * (size_t)a.tiles * kKv4Slots + slot0 + g;
        so[0] = p0[nt];
        so[8] = p1[nt];
      }
      raise = raise || fmaxf(p0[nt], p1[nt]) > m_ref[nt] + 8.f;
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx = fmaxf(p0[nt], p1[nt]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float m_new = fmaxf(m_ref[nt], mx);
        const float corr = m_ref[nt] == m_new ? 1.f : ex2(m_ref[nt] - m_new);
        m_ref[nt] = m_new;
        l[nt] *= corr;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[nt][i][k] *= corr;
      }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float m = m_ref[nt] == -INFINITY ? 0.f : m_ref[nt];
      p0[nt] = ex2(p0[nt] - m);
      p1[nt] = ex2(p1[nt] - m);
      l[nt] += p0[nt] + p1[nt];
      // column g of the B fragment: query g / 2, its weight or the remainder
      const int src = 8 * t + (g >> 1);
      const float v0 = __shfl_sync(0xffffffffu, p0[nt], src), v1 = __shfl_sync(0xffffffffu, p0[nt], src + 4);
      const float v2 = __shfl_sync(0xffffffffu, p1[nt], src), v3 = __shfl_sync(0xffffffffu, p1[nt], src + 4);
      const uint32_t h0 = pack2(v0, v1), h1 = pack2(v2, v3);
      if (g & 1) {
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
        pb[nt][0] = pack2(v0 - f0.x, v1 - f0.y);
        pb[nt][1] = pack2(v2 - f1.x, v3 - f1.y);
      } else {
        pb[nt][0] = h0;
        pb[nt][1] = h1;
      }
    }
    // ---- values: slots 2t, 2t+1 (par.x, par.y) and 2t+8, 2t+9 (par.z, par.w)
    uint4 par = lds128(d + 64 * C::CB + 32 * C::KPB + lane * 16);
    auto accumulate = [&](const uint4& vp) {
      constexpr int Q = D / 32;  // words per slot pair
      uint32_t w[2 * Q];
      if constexpr (D == 32) {
        const uint2 u = *reinterpret_cast<const uint2*>(d + 32 * C::CB + lane * 8);
        w[0] = u.x;
        w[1] = u.y;
      } else {
#pragma unroll
        for (int p = 0; p < Q / 2; ++p) {
          const uint4 u = lds128(d + 32 * C::CB + p * 512 + lane * 16);
          w[4 * p] = u.x;
          w[4 * p + 1] = u.y;
          w[4 * p + 2] = u.z;
          w[4 * p + 3] = u.w;
        }
      }
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        uint32_t e[4], f[4];
        dequant8(w[i], vp.x, vp.y, e);
        dequant8(w[Q + i], vp.z, vp.w, f);
        const uint32_t a0[4] = {e[0], e[1], f[0], f[1]}, a1[4] = {e[2], e[3], f[2], f[3]};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816(acc[nt][2 * i], a0, pb[nt][0], pb[nt][1]);
          mma_16816(acc[nt][2 * i + 1], a1, pb[nt][0], pb[nt][1]);
        }
      }
    };
    // slots that no query reads become zeros: their weight is zero, but an unread
    // NaN or infinity times zero would not be
    if (!full) {
      const int s = slot0 + 2 * t;
      auto live = [&](int x) { return x < lim_hi && !(x >= hole.x && x < hole.y); };
      const uint32_t k0 = (live(s) ? 0xFFFFu : 0u) | (live(s + 1) ? 0xFFFF0000u : 0u);
      const uint32_t k1 = (live(s + 8) ? 0xFFFFu : 0u) | (live(s + 9) ? 0xFFFF0000u : 0u);
      par.x &= k0, par.y &= k0, par.z &= k1, par.w &= k1;
    }
    if (!full && lim_lo != lim_hi) {
      // a slot that only some of the tile's queries read: where its group is not
      // finite it is left out of the products, and the queries that do read it
      // get NaN there (a lane's values of a slot all belong to one group)
      auto odd = [](uint32_t s, uint32_t m) {
        return (((s & 0x7C00u) == 0x7C00u || (m & 0x7C00u) == 0x7C00u) ? 1u : 0u) |
               (((s & 0x7C000000u) == 0x7C000000u || (m & 0x7C000000u) == 0x7C000000u) ? 2u : 0u);
      };
      const uint32_t b0 = odd(par.x, par.y), b1 = odd(par.z, par.w);
      uint32_t bad = (b0 << (2 * t)) | (b1 << (2 * t + 8));
      if (__any_sync(0xffffffffu, bad != 0u)) {
        const uint32_t k0 = (b0 & 1 ? 0u : 0xFFFFu) | (b0 & 2 ? 0u : 0xFFFF0000u);
        const uint32_t k1 = (b1 & 1 ? 0u : 0xFFFFu) | (b1 & 2 ? 0u : 0xFFFF0000u);
        par.x &= k0, par.y &= k0, par.z &= k1, par.w &= k1;
        bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
        bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int n = min(max(lim_q[nt] - slot0, 0), 16);  // the query reads the tile's first n slots
          if (bad & ((1u << n) - 1u))
#pragma unroll
            for (int i = 0; i < D / 16; ++i) acc[nt][i][0] = acc[nt][i][2] = __int_as_float(0x7FFFFFFF);
        }
      }
    }
    accumulate(par);
  }
  cp_wait<0>();
  __syncthreads();  // the rings are free: they take the warps' partials

  float* s_acc = reinterpret_cast<float*>(smem);  // [NW][NQ][D]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int i = 4 * nt + t;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], o);
    if (g == 0) {
      s_m[warp][i] = m_ref[nt];
      s_l[warp][i] = l[nt];
    }
    if (i < nq) {
      float* o = s_acc + ((size_t)warp * NQ + i) * D + g * (D / 8);
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        o[2 * x] = acc[nt][x][0] + acc[nt][x][1];
        o[2 * x + 1] = acc[nt][x][2] + acc[nt][x][3];
      }
    }
  }
  __syncthreads();
  // the CTA's partial of each query: maximum, sum, weighted values
  for (int i = warp; i < nq; i += NW) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w][i]);
    float f[NW], L = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {  // a warp without a finite maximum has summed nothing, or NaN
      f[w] = s_m[w][i] == -INFINITY ? (s_l[w][i] == 0.f ? 0.f : 1.f) : ex2(s_m[w][i] - M);
      L += s_l[w][i] * f[w];
    }
    for (int d = lane; d < D; d += 32) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v += s_acc[((size_t)w * NQ + i) * D + d] * f[w];
      s_part[i][2 + d] = v;
    }
    if (lane == 0) {
      s_part[i][0] = M;
      s_part[i][1] = L;
    }
  }
  // the splits' partials meet through the cluster's shared memory; every CTA
  // writes a slice of the output
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int ns = gridDim.x;
  if (ns > 1) {
    cluster.sync();
  } else {
    __syncthreads();
  }
  auto part = [&](int sp, int i) { return ns > 1 ? cluster.map_shared_rank(&s_part[i][0], sp) : &s_part[i][0]; };
  const float sink = a.sink ? a.sink[head] * 1.4426950408889634f : -INFINITY;
  for (int i = warp; i < nq; i += NW) {
    float M = sink;
    for (int sp = 0; sp < ns; ++sp) M = fmaxf(M, part(sp, i)[0]);
    float L = a.sink ? ex2(sink - M) : 0.f;
    auto factor = [&](const float* pp) {
      return pp[0] == -INFINITY ? (pp[1] == 0.f ? 0.f : 1.f) : ex2(pp[0] - M);
    };
    for (int sp = 0; sp < ns; ++sp) L += part(sp, i)[1] * factor(part(sp, i));
    const float inv = L == 0.f ? 0.f : 1.f / L;  // nothing to read: zeros
    const int d1 = (split + 1) * D / ns;
    for (int d = split * D / ns + lane; d < d1; d += 32) {
      float v = 0.f;
      for (int sp = 0; sp < ns; ++sp) v += part(sp, i)[2 + d] * factor(part(sp, i));
      store_elem(a.out, a.out_dtype, (long long)q_index(i) * D + d, v * inv);
    }
    if (lane == 0) {
      s_fin[i] = make_float2(M, inv);
      if (a.lse && split == 0) a.lse[q_index(i)] = s_fin[i];
    }
  }
  if (ns > 1) cluster.sync();  // a CTA keeps its partial until all slices are merged
  if (a.wts && a.kv_rstep) {
    // this CTA alone has these slots of the row: add its queries' weights in order
    __syncthreads();
    float* wt = a.wts + ((size_t)row * a.nh + head) * a.tiles * kKv4Slots;
    for (int x = threadIdx.x; x < (j1 - j0) * 16; x += NW * 32) {
      const int slot = tiles(j0 + (x >> 4)) * 16 + (x & 15);
      float add = 0.f;
      for (int i = 0; i < nq; ++i)
        add += ex2(a.scores[q_index(i) * (size_t)a.tiles * kKv4Slots + slot] - s_fin[i].x) * s_fin[i].y;
      if (add != 0.f) wt[slot] += add;
    }
  }
}

// The weights of a chunk's queries, which several CTAs hold: one thread per
// slot adds them in the tokens' order.
__global__ void k_kv4_track(const Kv4AttnArgs a, int tokens) {
  pdl_launch_dependents();
  pdl_wait();
  const int slot = blockIdx.x * blockDim.x + threadIdx.x, head = blockIdx.y, G = a.q_heads / a.nh;
  const int row = a.kv_row0;
  const int2 hole = a.hole[row];
  if (slot >= a.P + a.R || (slot >= hole.x && slot < hole.y)) return;
  float add = 0.f;
  for (int t = 0; t < tokens; ++t) {
    const int p = max(a.pos ? a.pos[t] : a.pos0 + t, 0);
    if (slot >= kv_limit(p, a.P, a.R)) continue;
    for (int g = 0; g < G; ++g) {
      const size_t qi = (size_t)t * a.q_heads + head * G + g;
      const float2 n = a.lse[qi];
      add += ex2(a.scores[qi * a.tiles * kKv4Slots + slot] - n.x) * n.y;
    }
  }
  if (add != 0.f) a.wts[((size_t)row * a.nh + head) * a.tiles * kKv4Slots + slot] += add;
}

template <int D, int NT>
static cudaError_t launch_attn4(const Kv4AttnArgs& a, int tokens, int nsplit, cudaStream_t st, bool pdl) {
  constexpr int part = kAttn4Warps * 4 * NT * D * 4, ring = kAttn4Warps * Attn4<D>::RING;
  const int queries = tokens * (a.q_heads / a.nh);
  const int z = a.kv_rstep ? tokens : (queries + 4 * NT - 1) / (4 * NT);
  return launch_kernel_cluster(k_kv4_attn<D, NT>, dim3(nsplit, a.nh, z), dim3(kAttn4Warps * 32),
                               (size_t)(part > ring ? part : ring), st, pdl, nsplit, a, queries);
}

template <int NT>
static cudaError_t launch_attn4(const Kv4AttnArgs& a, int tokens, int nsplit, cudaStream_t st, bool pdl) {
  switch (a.D) {
    case 32: return launch_attn4<32, NT>(a, tokens, nsplit, st, pdl);
    case 64: return launch_attn4<64, NT>(a, tokens, nsplit, st, pdl);
    case 128: return launch_attn4<128, NT>(a, tokens, nsplit, st, pdl);
    case 256: return launch_attn4<256, NT>(a, tokens, nsplit, st, pdl);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, int tokens, cudaStream_t st, bool pdl) {
  if (tokens <= 0) return cudaSuccess;
  const int G = a.q_heads / a.nh;
  // a second group of four queries costs registers: only where they exist
  const int nt = (a.kv_rstep ? G : tokens * G) > 4 ? 2 : 1;
  // splits: enough CTAs for two on every SM, each with a tile for every warp
  const int ctas = a.nh * (a.kv_rstep ? tokens : (tokens * G + 4 * nt - 1) / (4 * nt));
  int ns = (2 * a.n_sm + ctas - 1) / ctas;
  const int cap = (a.tiles + kAttn4Warps - 1) / kAttn4Warps;
  ns = ns > cap ? cap : ns;
  ns = ns > 8 ? 8 : ns < 1 ? 1 : ns;
  cudaError_t e = nt == 1 ? launch_attn4<1>(a, tokens, ns, st, pdl) : launch_attn4<2>(a, tokens, ns, st, pdl);
  if (e == cudaSuccess && a.wts && !a.kv_rstep)
    e = launch_kernel(k_kv4_track, dim3((a.P + a.R + 127) / 128, a.nh), dim3(128), 0, st, pdl, a, tokens);
  return e;
}

// ------------------------------------------------------------------ eviction
// Eight or four fp16 values, in one store where the address allows.
__device__ __forceinline__ void store16(__half* p, int wide, uint4 v) {
  if (wide) {
    *reinterpret_cast<uint4*>(p) = v;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = __ushort_as_half((unsigned short)(w[j >> 1] >> (16 * (j & 1))));
  }
}
__device__ __forceinline__ void store8(__half* p, int wide, uint2 v) {
  if (wide) {
    *reinterpret_cast<uint2*>(p) = v;
  } else {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = __ushort_as_half((unsigned short)(w[j >> 1] >> (16 * (j & 1))));
  }
}

// Order of the weights as unsigned integers; -0 counts as 0, a NaN as lowest.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (head, row, layer).  The key of the keep-th largest weight comes
// from three radix passes (11, 11, 10 bits; the first digit holds the exponent
// and two bits, which spreads weights over the bins; lanes with the same digit
// add once).  Then the kept entries move, lowest slot first, to the front of
// the destination row: live entries in blocks of the CTA's size are ranked by
// ballots, and the kept ones go through registers, several per warp at a time.
// A chunk is read before any of it is written and a kept entry never moves up,
// so source and destination may be the same row.  Bound by the scattered reads
// (a slot's values lie in 16-byte pieces of its tile) and the writes.
constexpr int kEvictThreads = 512;
constexpr int kEvictKeys = 4096;  // weights kept in shared memory between the passes
constexpr int kEvictPer = 4;      // entries of a warp in flight

template <int D>
__global__ void __launch_bounds__(kEvictThreads) k_kv4_evict(const Kv4EvictArgs a) {
  constexpr int T = kEvictThreads, NW = T / 32, NG = D / kKv4Group, E = kEvictPer, TB = kv4_tile_bytes(D);
  __shared__ uint32_t s_key[kEvictKeys];
  __shared__ int s_hist[2048];
  __shared__ int s_warp[2][NW];
  __shared__ int s_kept[T];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int head = blockIdx.x, r = blockIdx.y, l = blockIdx.z;
  const int layer = a.layer0 + l, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rs = a.src[r], rd = a.dst[r];
  const int2 hole = a.hole[(size_t)layer * a.MR + rs];
  const int gap = hole.y > hole.x ? hole.y - hole.x : 0;
  const int live = a.n - gap;  // live entry i is slot i, or i + gap behind the hole
  auto slot_of = [&](int i) { return gap && i >= hole.x ? i + gap : i; };
  const size_t SLt = (size_t)a.tiles * kKv4Slots;
  const float* ws = a.wts + (((size_t)layer * a.MR + rs) * a.nh + head) * SLt;
  float* wd = a.wts + (((size_t)layer * a.MR + rd) * a.nh + head) * SLt;
  const bool cached = live <= kEvictKeys;
  if (cached)
    for (int i = tid; i < live; i += T) s_key[i] = weight_key(ws[slot_of(i)]);
  auto key_of = [&](int i) { return cached ? s_key[i] : weight_key(ws[slot_of(i)]); };
  // the keep - protect largest of the entries behind the protected ones
  if (tid == 0) {
    s_prefix = 0u;
    s_need = a.keep - a.protect;
  }
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < 2048; i += T) s_hist[i] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    const int need = s_need;
    for (int i0 = a.protect; i0 < live; i0 += T) {
      const int i = i0 + tid;
      const uint32_t k = i < live ? key_of(i) : 0u;
      const bool in = i < live && (pass == 0 || (k >> (shift + bits)) == (prefix >> (shift + bits)));
      const uint32_t digit = in ? (k >> shift) & ((1u << bits) - 1u) : 0xFFFFFFFFu;
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      if (in && lane == __ffs(same) - 1) atomicAdd(&s_hist[digit], __popc(same));
    }
    __syncthreads();
    // thread t holds the four bins below 2048 - 4t: counts of everything above them
    int c[4], sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += c[j] = s_hist[2047 - 4 * tid - j];
    int up = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    if (lane == 31) s_warp[0][warp] = up;
    __syncthreads();
    int above = up - sum;
    for (int w = 0; w < warp; ++w) above += s_warp[0][w];
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // the bin that holds the need-th largest
      if (above < need && above + c[j] >= need) {
        s_prefix = prefix | ((uint32_t)(2047 - 4 * tid - j) << shift);
        s_need = need - above;
      }
      above += c[j];
    }
    __syncthreads();
  }
  // entries equal to the threshold stay while there is room, lowest slot first;
  // nothing beyond the protected ones stays when none is needed
  const bool some = a.keep > a.protect;
  const uint32_t kth = s_prefix;
  const int ties = some ? s_need : 0;

  const uint8_t* src = a.kv4 + (((size_t)layer * a.MR + rs) * 2 * a.nh + head) * a.tiles * TB;
  uint8_t* dst = a.kv4 + (((size_t)layer * a.MR + rd) * 2 * a.nh + head) * a.tiles * TB;
  const size_t voff = (size_t)a.nh * a.tiles * TB;
  const size_t out0 = (((size_t)l * a.rows + r) * a.nh + head) * a.keep;
  int done = 0, tied = 0;
  for (int i0 = 0; i0 < live && done < a.keep; i0 += T) {
    const int i = i0 + tid;
    bool eq = false, keep = false;
    if (i < live) {
      if (i < a.protect) {
        keep = true;
      } else if (some) {
        const uint32_t k = key_of(i);
        eq = k == kth;
        keep = k > kth;
      }
    }
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t eqs = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_warp[0][warp] = __popc(eqs);
    __syncthreads();
    int before = tied + __popc(eqs & below);
    for (int w = 0; w < NW; ++w) {
      if (w < warp) before += s_warp[0][w];
      tied += s_warp[0][w];
    }
    keep = keep || (eq && before < ties);
    const uint32_t keeps = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) s_warp[1][warp] = __popc(keeps);
    __syncthreads();
    int at = __popc(keeps & below), count = 0;
    for (int w = 0; w < NW; ++w) {
      if (w < warp) at += s_warp[1][w];
      count += s_warp[1][w];
    }
    if (keep) s_kept[at] = slot_of(i);
    __syncthreads();
    for (int c0 = 0; c0 < count; c0 += NW * E) {
      uint32_t kw[E], kpar[E];
      uint16_t vq[E][D == 256 ? 2 : 1], vpar[E];
      float wt[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = c0 + e * NW + warp;
        if (c < count) {
          const int ss = s_kept[c], s = ss & 15;
          const uint8_t* kp = src + (size_t)(ss >> 4) * TB;
          const uint8_t* vp = kp + voff;
          if (lane < D / 8) kw[e] = *reinterpret_cast<const uint32_t*>(kp + kv4_k_word(D, s, lane));
          if (lane < NG) kpar[e] = *reinterpret_cast<const uint32_t*>(kp + kv4_k_param(D, s, lane));
          if (lane < D / 4) vq[e][0] = *reinterpret_cast<const uint16_t*>(vp + kv4_v_quad(D, s, lane));
          if constexpr (D == 256) vq[e][1] = *reinterpret_cast<const uint16_t*>(vp + kv4_v_quad(D, s, lane + 32));
          if (lane < 2 * NG) vpar[e] = *reinterpret_cast<const uint16_t*>(vp + kv4_v_param(D, s, lane >> 1, lane & 1));
          if (lane == 0) wt[e] = ws[ss];
        }
      }
      __syncthreads();  // the chunk is in registers
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = c0 + e * NW + warp;
        if (c < count) {
          const int ds = done + c, s = ds & 15;
          uint8_t* kp = dst + (size_t)(ds >> 4) * TB;
          uint8_t* vp = kp + voff;
          if (lane < D / 8) *reinterpret_cast<uint32_t*>(kp + kv4_k_word(D, s, lane)) = kw[e];
          if (lane < NG) *reinterpret_cast<uint32_t*>(kp + kv4_k_param(D, s, lane)) = kpar[e];
          if (lane < D / 4) *reinterpret_cast<uint16_t*>(vp + kv4_v_quad(D, s, lane)) = vq[e][0];
          if constexpr (D == 256) *reinterpret_cast<uint16_t*>(vp + kv4_v_quad(D, s, lane + 32)) = vq[e][1];
          if (lane < 2 * NG) *reinterpret_cast<uint16_t*>(vp + kv4_v_param(D, s, lane >> 1, lane & 1)) = vpar[e];
          if (lane == 0) {
            wd[ds] = wt[e];
            if (a.kept) a.kept[out0 + ds] = s_kept[c];
          }
          if (a.k_val) {  // word w belongs to group w / 4
            const uint32_t p = __shfl_sync(0xffffffffu, kpar[e], lane >> 2);
            const uint32_t sc = __byte_perm(p, 0, 0x1010), lo = __byte_perm(p, 0, 0x3232);
            uint32_t x[4];
            dequant8(kw[e], sc, lo, x);
            if (lane < D / 8)
              store16(a.k_val + (out0 + ds) * D + 8 * lane, a.wide, make_uint4(x[0], x[1], x[2], x[3]));
          }
          if (a.v_val) {  // quad i belongs to group i / 8
#pragma unroll
            for (int h = 0; h < (D == 256 ? 2 : 1); ++h) {
              const int grp = (lane + 32 * h) >> 3;
              const uint32_t sc = __shfl_sync(0xffffffffu, (uint32_t)vpar[e], 2 * grp) * 0x10001u;
              const uint32_t lo = __shfl_sync(0xffffffffu, (uint32_t)vpar[e], 2 * grp + 1) * 0x10001u;
              const uint32_t q = vq[e][h];
              uint32_t x[4];
              // nibbles 0, 1 to one word's halves and 2, 3 to the other's
              dequant8((q & 0xFu) | ((q & 0xF0u) << 12) | ((q & 0xF00u) >> 4) | ((q & 0xF000u) << 8), sc, lo, x);
              if (lane + 32 * h < D / 4)
                store8(a.v_val + (out0 + ds) * D + 4 * (lane + 32 * h), a.wide, make_uint2(x[0], x[1]));
            }
          }
        }
      }
      __syncthreads();  // the next chunk's reads follow these writes
    }
    done += count;
  }
  for (int i = a.keep + tid; i < a.n; i += T) wd[i] = 0.f;
  if (!a.in_place && head == 0 && tid == 0)
    a.hole[(size_t)layer * a.MR + rd] = a.keep < a.n ? make_int2(a.keep, a.n) : make_int2(0, 0);
}

// The holes of rows that were their own source, whose heads all had to read them.
__global__ void k_kv4_hole(const Kv4EvictArgs a) {
  const int r = threadIdx.x, l = blockIdx.x;
  if (r < a.rows)
    a.hole[(size_t)(a.layer0 + l) * a.MR + a.dst[r]] = a.keep < a.n ? make_int2(a.keep, a.n) : make_int2(0, 0);
}

cudaError_t launch_kv4_evict(const Kv4EvictArgs& args, cudaStream_t st) {
  Kv4EvictArgs a = args;
  a.in_place = 0;
  for (int i = 0; i < a.rows; ++i) a.in_place |= a.src[i] == a.dst[i];
  a.wide = ((uintptr_t)a.k_val | (uintptr_t)a.v_val) % 16 == 0;
  const dim3 grid(a.nh, a.rows, a.layers);
  switch (a.D) {
    case 32: k_kv4_evict<32><<<grid, kEvictThreads, 0, st>>>(a); break;
    case 64: k_kv4_evict<64><<<grid, kEvictThreads, 0, st>>>(a); break;
    case 128: k_kv4_evict<128><<<grid, kEvictThreads, 0, st>>>(a); break;
    case 256: k_kv4_evict<256><<<grid, kEvictThreads, 0, st>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.in_place) return e;
  k_kv4_hole<<<a.layers, kKv4MaxRows, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t init_kv4_attributes() {
  cudaError_t e = cudaSuccess;
#define UOCR_A(D_)                                              \
  if (e == cudaSuccess) e = allow_max_dyn_smem(k_kv4_attn<D_, 1>); \
  if (e == cudaSuccess) e = allow_max_dyn_smem(k_kv4_attn<D_, 2>);
  UOCR_A(32) UOCR_A(64) UOCR_A(128) UOCR_A(256)
#undef UOCR_A
  return e;
}

}  // namespace uocr
