// The 4-bit KV cache: rotary positions and the append, attention over the
// entries, and the eviction of the entries that attention uses least.
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

// Element d of a rotated vector: (x, y) -> (x c - y s, y c + x s), the products
// and the sum each rounded to fp32.
__device__ __forceinline__ float rotated(const void* p, int dtype, long long base, int d, const Kv4AppendArgs& a,
                                         const float2* cs) {
  const float x = load_elem(p, dtype, base + d);
  if (!a.rotate || d >= a.rope_dims) return x;
  const int half = a.rope_dims >> 1;
  int j, other;
  bool lo;
  if (a.rope_layout == 0) {
    lo = d < half;
    j = lo ? d : d - half;
    other = lo ? d + half : d - half;
  } else {
    lo = !(d & 1);
    j = d >> 1;
    other = d ^ 1;
  }
  const float y = load_elem(p, dtype, base + other);
  const float2 r = cs[j];
  return lo ? __fsub_rn(__fmul_rn(x, r.x), __fmul_rn(y, r.y)) : __fadd_rn(__fmul_rn(x, r.x), __fmul_rn(y, r.y));
}

// One CTA per token.  A thread takes eight dimensions of a key or value
// vector, four neighbouring lanes a group of 32.
__global__ void __launch_bounds__(256) k_kv4_append(const Kv4AppendArgs a) {
  __shared__ float2 s_cs[128];
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
    for (int j = threadIdx.x; j < (a.rope_dims >> 1); j += blockDim.x) {
      double sn, cs;
      sincos_taylor((double)p * a.inv_freq[j], sn, cs);
      s_cs[j] = make_float2((float)(a.amp * cs), (float)(a.amp * sn));
    }
    __syncthreads();
  }
  if (a.q_out)
    for (int i = threadIdx.x; i < a.q_heads * D; i += blockDim.x)
      a.q_out[(size_t)t * a.q_heads * D + i] = rotated(a.q, a.dtype, t * a.ldq + (i / D) * D, i % D, a, s_cs);

  const int wpv = D / 8;  // words per vector
  uint8_t* row4 = a.kv4 + (size_t)row * 2 * a.nh * a.tiles * kv4_tile_bytes(D);
  const int tile = slot >> 4, s = slot & 15;
  const int total = 2 * a.nh * wpv;  // a multiple of 4
  for (int i0 = 0; i0 < total; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    const bool in = i < total;
    const int vec = in ? i / wpv : 0, w = in ? i % wpv : 0;
    const int kv = vec >= a.nh, head = kv ? vec - a.nh : vec;
    float x[8];
    float mn = INFINITY, mx = -INFINITY;
    bool ok = true;
    if (in) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = kv ? load_elem(a.v, a.dtype, t * a.ldv + head * a.lhk + 8 * w + j)
                  : rotated(a.k, a.dtype, t * a.ldk + head * a.lhk, 8 * w + j, a, s_cs);
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
#pragma unroll
      for (int j = 0; j < 8; ++j) val[j] = kv4_value(c[j], sc, lo);
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
  return launch_kernel(k_kv4_append, dim3(tokens), dim3(256), 0, st, pdl, a);
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
// One CTA per (query head, token): every warp takes slots in turn, a lane
// eight dimensions, and keeps an online softmax; the warps merge at the end.
__global__ void __launch_bounds__(128) k_kv4_attn(const Kv4AttnArgs a) {
  constexpr int NW = 4;
  __shared__ float s_m[NW], s_l[NW], s_acc[NW][256];
  pdl_launch_dependents();
  pdl_wait();
  const int qh = blockIdx.x, t = blockIdx.y, D = a.D, W = D / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = qh / (a.q_heads / a.nh), row = a.kv_row0 + t * a.kv_rstep;
  int p = a.pos ? a.pos[t] : a.pos0 + t;
  const int2 hole = a.hole[row];
  if (p < 0 || (hole.y > hole.x && p < hole.y)) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusPosition);
    p = max(p, 0);
  }
  const int lim = kv_limit(p, a.P, a.R);
  const uint8_t* kt = a.kv4 + (size_t)(row * 2 * a.nh + head) * a.tiles * kv4_tile_bytes(D);
  const uint8_t* vt = kt + (size_t)a.nh * a.tiles * kv4_tile_bytes(D);
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = lane < W ? a.q[((size_t)t * a.q_heads + qh) * D + 8 * lane + j] * a.scale : 0.f;
  float m = -INFINITY, l = 0.f, acc[8] = {};
  for (int slot = warp; slot < lim; slot += NW) {
    if (slot >= hole.x && slot < hole.y) continue;
    const int s = slot & 15;
    const size_t off = (size_t)(slot >> 4) * kv4_tile_bytes(D);
    float d = 0.f;
    if (lane < W) {
      __half x[8];
      key_values(kt + off, D, s, lane, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) d = fmaf(q[j], __half2float(x[j]), d);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    const float mn = fmaxf(m, d);
    const float corr = m == -INFINITY ? 0.f : __expf(m - mn);
    const float w = mn == -INFINITY ? 0.f : __expf(d - mn);
    l = l * corr + w;
    m = mn;
    if (lane < W) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        __half x[4];
        value_values(vt + off, D, s, 2 * lane + h, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[4 * h + j] = fmaf(w, __half2float(x[j]), acc[4 * h + j] * corr);
      }
    }
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  if (lane < W)
#pragma unroll
    for (int j = 0; j < 8; ++j) s_acc[warp][8 * lane + j] = acc[j];
  __syncthreads();
  float M = a.sink ? a.sink[head] : -INFINITY;
  for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w]);
  float L = a.sink ? __expf(a.sink[head] - M) : 0.f;
  for (int w = 0; w < NW; ++w)
    if (s_l[w] != 0.f) L += s_l[w] * __expf(s_m[w] - M);
  const float inv = L != 0.f ? 1.f / L : 0.f;  // nothing to read: the output is zero
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float v = 0.f;
    for (int w = 0; w < NW; ++w)
      if (s_l[w] != 0.f) v += s_acc[w][d] * __expf(s_m[w] - M);
    store_elem(a.out, a.out_dtype, ((long long)t * a.q_heads + qh) * D + d, v * inv);
  }
  if (a.lse && threadIdx.x == 0) a.lse[(size_t)t * a.q_heads + qh] = make_float2(M, inv);
}

// Accumulate the softmax weights that the attention gave: one warp per (slot,
// head, row) adds the weights of every query of the row in order.
__global__ void k_kv4_track(const Kv4AttnArgs a, int tokens) {
  pdl_launch_dependents();
  pdl_wait();
  const int slot = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int head = blockIdx.y, D = a.D, W = D / 8, G = a.q_heads / a.nh;
  const int row = a.kv_row0 + blockIdx.z * a.kv_rstep;
  const int t0 = a.kv_rstep ? blockIdx.z : 0, t1 = a.kv_rstep ? t0 + 1 : tokens;
  const int2 hole = a.hole[row];
  if (slot >= a.P + a.R || (slot >= hole.x && slot < hole.y)) return;
  const uint8_t* kt = a.kv4 + ((size_t)(row * 2 * a.nh + head) * a.tiles + (slot >> 4)) * kv4_tile_bytes(D);
  __half x[8];
  if (lane < W) key_values(kt, D, slot & 15, lane, x);
  float add = 0.f;
  for (int t = t0; t < t1; ++t) {
    const int p = max(a.pos ? a.pos[t] : a.pos0 + t, 0);
    if (slot >= kv_limit(p, a.P, a.R)) continue;
    for (int g = 0; g < G; ++g) {
      const size_t qi = (size_t)t * a.q_heads + head * G + g;
      float d = 0.f;
      if (lane < W)
#pragma unroll
        for (int j = 0; j < 8; ++j) d = fmaf(a.q[qi * D + 8 * lane + j] * a.scale, __half2float(x[j]), d);
#pragma unroll
      for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      const float2 n = a.lse[qi];
      add += __expf(d - n.x) * n.y;
    }
  }
  if (lane == 0 && add != 0.f) a.wts[((size_t)row * a.nh + head) * a.tiles * kKv4Slots + slot] += add;
}

cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, int tokens, cudaStream_t st, bool pdl) {
  if (tokens <= 0) return cudaSuccess;
  cudaError_t e = launch_kernel(k_kv4_attn, dim3(a.q_heads, tokens), dim3(128), 0, st, pdl, a);
  if (e == cudaSuccess && a.wts)
    e = launch_kernel(k_kv4_track, dim3((a.P + a.R + 7) / 8, a.nh, a.kv_rstep ? tokens : 1), dim3(256), 0, st, pdl, a,
                      tokens);
  return e;
}

// ------------------------------------------------------------------ eviction
// Order of the weights as unsigned integers; -0 counts as 0, a NaN as lowest.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (head, row, layer): the key of the keep-th largest weight by four
// 8-bit radix passes, then the kept entries move, lowest slot first, to the
// front of the destination row.  A chunk of kept entries is read into registers
// before any of it is written, and a kept entry never moves up, so source and
// destination may be the same row.
__global__ void __launch_bounds__(256) k_kv4_evict(const Kv4EvictArgs a) {
  __shared__ int s_hist[256], s_scan[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int head = blockIdx.x, r = blockIdx.y, l = blockIdx.z, D = a.D, NG = D / kKv4Group;
  const int layer = a.layer0 + l, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rs = a.src[r], rd = a.dst[r];
  const int2 hole = a.hole[(size_t)layer * a.MR + rs];
  const int gap = hole.y > hole.x ? hole.y - hole.x : 0;
  const int live = a.n - gap;  // live entry i is slot i, or i + gap behind the hole
  auto slot_of = [&](int i) { return gap && i >= hole.x ? i + gap : i; };
  const size_t SLt = (size_t)a.tiles * kKv4Slots;
  const float* ws = a.wts + (((size_t)layer * a.MR + rs) * a.nh + head) * SLt;
  float* wd = a.wts + (((size_t)layer * a.MR + rd) * a.nh + head) * SLt;
  auto key_of = [&](int i) { return weight_key(ws[slot_of(i)]); };
  // the keep - protect largest of the entries behind the protected ones
  if (tid == 0) {
    s_prefix = 0u;
    s_need = a.keep - a.protect;
  }
  __syncthreads();
  for (int shift = 24; shift >= 0; shift -= 8) {
    s_hist[tid] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    for (int i = a.protect + tid; i < live; i += 256) {
      const uint32_t k = key_of(i);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&s_hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int need = s_need, b = 255;
      for (; b > 0 && s_hist[b] < need; --b) need -= s_hist[b];
      s_need = need;
      s_prefix = prefix | ((uint32_t)b << shift);
    }
    __syncthreads();
  }
  const uint32_t kth = s_prefix;
  const int ties = s_need;  // entries equal to the threshold that stay, lowest slot first
  // move: blocks of 256 live entries, kept ones in order, eight entries at a time
  const uint8_t* src = a.kv4 + ((size_t)layer * a.MR + rs) * 2 * a.nh * a.tiles * kv4_tile_bytes(D);
  uint8_t* dst = a.kv4 + ((size_t)layer * a.MR + rd) * 2 * a.nh * a.tiles * kv4_tile_bytes(D);
  const size_t voff = (size_t)a.nh * a.tiles * kv4_tile_bytes(D);
  src += (size_t)head * a.tiles * kv4_tile_bytes(D);
  dst += (size_t)head * a.tiles * kv4_tile_bytes(D);
  const size_t out0 = (((size_t)l * a.rows + r) * a.nh + head) * a.keep;
  __shared__ int s_kept[256];
  __shared__ int s_n;
  int done = 0, tied = 0;
  for (int i0 = 0; i0 < live; i0 += 256) {
    const int i = i0 + tid;
    uint32_t k = 0;
    bool eq = false, keep = false;
    if (i < live) {
      if (i < a.protect) {
        keep = true;
      } else {
        k = key_of(i);
        eq = k == kth;
        keep = k > kth;
      }
    }
    // rank among the ties of this block
    s_scan[tid] = eq;
    __syncthreads();
    int before = 0, all = 0;
    for (int j = 0; j < 256; ++j) {
      const int e = s_scan[j];
      if (j < tid) before += e;
      all += e;
    }
    if (eq && tied + before < ties) keep = true;
    tied += all;
    __syncthreads();
    s_scan[tid] = keep;
    __syncthreads();
    int at = 0, count = 0;
    for (int j = 0; j < 256; ++j) {
      const int e = s_scan[j];
      if (j < tid) at += e;
      count += e;
    }
    if (keep) s_kept[at] = i;
    if (tid == 0) s_n = count;
    __syncthreads();
    for (int c0 = 0; c0 < s_n; c0 += 8) {
      const bool in = c0 + warp < s_n;
      const int ss = in ? slot_of(s_kept[c0 + warp]) : 0, ds = done + c0 + warp;
      const uint8_t* kp = src + (size_t)(ss >> 4) * kv4_tile_bytes(D);
      const uint8_t* vp = kp + voff;
      uint32_t kw = 0, kpar = 0;
      uint16_t vq[2] = {}, vpar = 0;
      float wt = 0.f;
      if (in) {
        const int s = ss & 15;
        if (lane < D / 8) kw = *reinterpret_cast<const uint32_t*>(kp + kv4_k_word(D, s, lane));
        if (lane < NG) kpar = *reinterpret_cast<const uint32_t*>(kp + kv4_k_param(D, s, lane));
        if (lane < D / 4) vq[0] = *reinterpret_cast<const uint16_t*>(vp + kv4_v_quad(D, s, lane));
        if (lane + 32 < D / 4) vq[1] = *reinterpret_cast<const uint16_t*>(vp + kv4_v_quad(D, s, lane + 32));
        if (lane < 2 * NG) vpar = *reinterpret_cast<const uint16_t*>(vp + kv4_v_param(D, s, lane >> 1, lane & 1));
        wt = ws[ss];
        if (lane == 0 && a.kept) a.kept[out0 + ds] = ss;
        const size_t o = (out0 + ds) * D;
        if (a.k_val && lane < D / 8) {
          __half x[8];
          key_values(kp, D, s, lane, x);
#pragma unroll
          for (int j = 0; j < 8; ++j) a.k_val[o + 8 * lane + j] = x[j];
        }
        if (a.v_val)
          for (int w = lane; w < D / 4; w += 32) {
            __half x[4];
            value_values(vp, D, s, w, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) a.v_val[o + 4 * w + j] = x[j];
          }
      }
      __syncthreads();  // the chunk is in registers
      if (in) {
        const int s = ds & 15;
        uint8_t* kq = dst + (size_t)(ds >> 4) * kv4_tile_bytes(D);
        uint8_t* vd = kq + voff;
        if (lane < D / 8) *reinterpret_cast<uint32_t*>(kq + kv4_k_word(D, s, lane)) = kw;
        if (lane < NG) *reinterpret_cast<uint32_t*>(kq + kv4_k_param(D, s, lane)) = kpar;
        if (lane < D / 4) *reinterpret_cast<uint16_t*>(vd + kv4_v_quad(D, s, lane)) = vq[0];
        if (lane + 32 < D / 4) *reinterpret_cast<uint16_t*>(vd + kv4_v_quad(D, s, lane + 32)) = vq[1];
        if (lane < 2 * NG) *reinterpret_cast<uint16_t*>(vd + kv4_v_param(D, s, lane >> 1, lane & 1)) = vpar;
        if (lane == 0) wd[ds] = wt;
      }
      __syncthreads();
    }
    done += s_n;
    __syncthreads();
  }
  for (int i = a.keep + tid; i < a.n; i += 256) wd[i] = 0.f;
}

// The destination rows' holes, once every head has moved.
__global__ void k_kv4_hole(const Kv4EvictArgs a) {
  const int r = threadIdx.x, l = blockIdx.x;
  if (r < a.rows)
    a.hole[(size_t)(a.layer0 + l) * a.MR + a.dst[r]] = a.keep < a.n ? make_int2(a.keep, a.n) : make_int2(0, 0);
}

cudaError_t launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t st) {
  k_kv4_evict<<<dim3(a.nh, a.rows, a.layers), 256, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_kv4_hole<<<a.layers, kKv4MaxRows, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t init_kv4_attributes() { return cudaSuccess; }

}  // namespace uocr
