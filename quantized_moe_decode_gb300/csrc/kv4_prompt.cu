// Attention of a prompt over the 4-bit cache: chunks of many tokens, on the fifth
// generation tensor cores.
//
// An item is 128 queries of one head (tokens times the heads that share the cache
// head); it goes through the slots in blocks of four 16-slot tiles, each
// dequantised once for all of them:
//   four warps dequantise a block into the K-major operands of shared memory,
//     keys [64 slots][D] and values transposed [D][64 slots] (a tile's words hold
//     eight dimensions of a slot, or one dimension of a slot pair, side by side);
//   one thread issues S = Q K^T (M 128, N 64) and O += P V (M 128, N D) into
//     tensor memory, S twice buffered;
//   eight warps, two threads per query with half of the block's scores each, read
//     S, keep the softmax (the pair exchanges its maxima), write P to shared
//     memory, and rescale O in tensor memory when the maximum has grown by 2^8,
//     which almost never happens.
// As in the decode kernel queries and weights are pairs of fp16 numbers (value and
// remainder), here as two products, which keeps about 22 bits; sums are fp32.
// The call's blocks are cut into equal runs, one per SM, an item's start counting
// as kPromptStart blocks; an item that several runs share leaves partials, which a
// second kernel merges.
// What it cannot do without are those products (4 M N K of them per block and
// pass); the softmax of 64 x 128 scores takes about as long on the other pipes.
#include "kv4_device.cuh"
#include "launch.h"
#include "tc_common.cuh"

namespace uocr {

constexpr int kPromptThreads = 416;  // warps 0-7 softmax, 8-11 dequantising, 12 issues
constexpr int kPromptStart = 4;      // what an item's start and end take, in blocks
constexpr int kPromptMaxZ = 2048;    // query tiles of a call that is cut into runs

template <int D>
struct Prompt4 {
  static constexpr int M = 128, N = 64;
  static constexpr int QL = 128, QS = D / 8 * 128;        // bytes between core matrices along K and M/N: queries,
  static constexpr int KL = 144, KS = D / 8 * KL;         // keys (padded: two bank passes instead of four),
  static constexpr int VL = 128, VS = N / 8 * 128 + 16;   // values (padded likewise),
  static constexpr int PL = 128, PS = N / 8 * 128;        // weights
  static constexpr int QB = M / 8 * QS, KB = N / 8 * KS, VB = D / 8 * VS, PB = M / 8 * PS;
  static constexpr int Q = 0, K = 2 * QB, V = K + 2 * KB, P = V + 2 * VB, SMEM = P + 2 * PB;
  static constexpr int COLS = 128 + D <= 256 ? 256 : 512;  // tensor memory columns: S, S, O
  static constexpr int O = 128;
};

struct PromptBars {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full, pv_done, all_done;
};

// Bounded wait: gives up after kSpinLimit polls, or when another role has.
__device__ __forceinline__ bool prompt_wait(uint64_t* bar, uint32_t parity, volatile int* dead) {
  for (uint32_t i = 0; i < kSpinLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 63u && *dead) return false;
  }
  *dead = 1;
  return false;
}

__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Blocks of query tile z of a chunk (positions rise and do not wrap, so that a
// query at position p reads p + 1 slots but the evicted ones).
__device__ __forceinline__ int prompt_blocks(const Kv4AttnArgs& a, int z, int n_queries, int G, int2 hole) {
  const int last = min((z + 1) * 128, n_queries) - 1;
  return (TileList(token_limit(a, last / G, hole, false), hole).count + 3) >> 2;
}

// A thread waits at a barrier of the softmax warps.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Cumulated blocks of the query tiles, kPromptStart more for each, for the runs
// (every thread of a CTA).  An item's blocks follow its start in the list.
__device__ __forceinline__ int prompt_runs(const Kv4AttnArgs& a, int n_queries, int n_z, int* cum, Attn4Runs& r) {
  const int2 hole = a.hole[a.kv_row0];
  const int G = a.q_heads / a.nh, lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    int before = 0;
    if (lane == 0) cum[0] = 0;
    for (int z0 = 0; z0 < n_z; z0 += 32) {
      const int z = z0 + lane;
      int up = z < n_z ? prompt_blocks(a, z, n_queries, G, hole) + kPromptStart : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += v;
      }
      if (z < n_z) cum[z + 1] = before + up;
      before += __shfl_sync(0xffffffffu, up, 31);
    }
  }
  __syncthreads();
  r.cum = cum;
  r.nh = a.nh;
  r.uniform = 0;
  const int total = cum[n_z] * a.nh;
  r.per = (total + a.n_runs - 1) / a.n_runs;
  return total;
}

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1) k_kv4_prompt(const Kv4AttnArgs a, int n_queries, int n_z) {
  using C = Prompt4<D>;
  constexpr int W = D / 32;  // words of a lane per slot (keys) or slot pair (values)
  constexpr uint32_t IDESC_S = idesc_f16(128, C::N), IDESC_O = idesc_f16(128, D);
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ PromptBars bars;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_dead;
  __shared__ unsigned s_bad[2][4][8];  // by block parity, tile, chunk of dimensions: slots whose group is not finite
  __shared__ int s_cum[kPromptMaxZ + 1];
  __shared__ float s_cq[128];
  __shared__ float s_pair[2][2][128];  // the pair's maxima, by block parity; its sums and NaN masks at the end
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int G = a.q_heads / a.nh, row = a.kv_row0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.k_full[i], 4);
      mbar_init(&bars.v_full[i], 4);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_empty[i], 1);
      mbar_init(&bars.s_full[i], 1);
    }
    mbar_init(&bars.p_full, 8);
    mbar_init(&bars.pv_done, 1);
    mbar_init(&bars.all_done, 1);
    fence_mbar_init();
    s_dead = 0;
  }
  if (warp == 12) {
    tmem_alloc(&s_tmem, C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  pdl_wait();
  pdl_launch_dependents();
  const int2 hole = a.hole[row];
  Attn4Runs runs;
  int at = 0, end = 1, z, head;
  if (a.n_runs) {
    const int total = prompt_runs(a, n_queries, n_z, s_cum, runs);
    at = min((int)blockIdx.x * runs.per, total);
    end = min(total, at + runs.per);
    int lo = 0, hi = n_z;  // the query tile that holds block `at`: the last with start <= at
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_cum[mid] * a.nh <= at) lo = mid; else hi = mid;
    }
    z = lo;
    head = at < end ? (at - s_cum[z] * a.nh) / max(runs.tiles(z), 1) : 0;
  } else {
    z = n_z - 1 - blockIdx.x / a.nh;  // a chunk's last tokens read most: first
    head = blockIdx.x % a.nh;
  }
  const size_t v_off = (size_t)a.nh * a.tiles * kv4_tile_bytes(D);

  int it = 0;  // blocks so far: the buffers' and barriers' phases
  const int run0 = at;
  while (at < end) {
    const int u0 = z * 128, nq = min(128, n_queries - u0);
    const int lim_lo = token_limit(a, u0 / G, hole, false), lim_hi = token_limit(a, (u0 + nq - 1) / G, hole, false);
    const TileList tiles(lim_hi, hole);
    const int blocks = (tiles.count + 3) >> 2;
    int b0 = 0, b1 = blocks;
    bool inside = false;  // the item begins inside the run: the run's second partial
    if (a.n_runs) {
      const int s = runs.start(z, head) + kPromptStart;
      b0 = max(at - s, 0);
      b1 = max(min(end - s, blocks), 0);
      inside = s > run0;
      at = s + b1 < end && b1 == blocks ? s + b1 : end;
    } else {
      at = end;
    }
    if (b0 >= b1) {  // the start only: the blocks are the next run's
      if (++head == a.nh) {
        head = 0;
        ++z;
      }
      continue;
    }
    const bool whole = b0 == 0 && b1 == blocks;
    auto first_slot = [&](int j) { return j < tiles.count ? tiles(j) * 16 : 0x7FFFFF00; };
    auto is_full = [&](int s) { return s + 16 <= lim_lo && (hole.y <= hole.x || s + 16 <= hole.x || s >= hole.y); };

    // ---- queries: D / 4 lanes to a row, four dimensions each (the last item's
    // products are done)
    if (warp < 8) {
      constexpr int LR = D / 4, RW = 32 / LR, PASSES = 16 / RW;  // lanes of a row, rows of a warp's pass
      const int c = (lane % LR) * 4;
      float4 q[PASSES];
      int tok = (u0 + warp * 16 + lane / LR) / G, rem = u0 + warp * 16 + lane / LR - tok * G;
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (warp * 16 + i * RW + lane / LR < nq) {
          const float* p = a.q + ((size_t)tok * a.q_heads + head * G + rem) * D + c;
          q[i] = a.q_wide ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], p[1], p[2], p[3]);
        }
        rem += RW;
        while (rem >= G) {
          rem -= G;
          ++tok;
        }
      }
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int r = warp * 16 + i * RW + lane / LR;
        float4 x = q[i];
        float mx = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
        for (int o = 1; o < LR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        // 2^-e with e the exponent of the largest magnitude (0 and infinities stay)
        const int e = mx > 0.f && mx < INFINITY ? min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 100) : 0;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        if (c == 0) s_cq[r] = a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23);
        x.x *= down, x.y *= down, x.z *= down, x.w *= down;
        const uint32_t h0 = pack2(x.x, x.y), h1 = pack2(x.z, x.w);
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
        unsigned char* o = smem + C::Q + (r >> 3) * C::QS + (c >> 3) * C::QL + (r & 7) * 16 + (c & 7) * 2;
        *reinterpret_cast<uint2*>(o) = make_uint2(h0, h1);
        *reinterpret_cast<uint2*>(o + C::QB) = make_uint2(pack2(x.x - f0.x, x.y - f0.y), pack2(x.z - f1.x, x.w - f1.y));
      }
      fence_proxy_async_smem();
    }
    __syncthreads();

    if (warp >= 8 && warp < 12) {  // ---------------- dequantise: tile n of every block
      const int n = warp - 8;
      const uint8_t* kt = a.kv4 + ((size_t)row * 2 * a.nh + head) * a.tiles * kv4_tile_bytes(D);
      const int kp_off = 8 * D + (g * W + t * W / 4) * 8;
      const int vp_off = 8 * D + ((g * D / 256) * 4 + t) * 16;
      uint32_t kc[2 * W], vc[2 * W];
      uint2 kpar = make_uint2(0u, 0u);
      uint4 vpar = make_uint4(0u, 0u, 0u, 0u);
      auto load_codes = [&](const uint8_t* p, uint32_t (&w)[2 * W]) {
        if constexpr (D == 32) {
          const uint2 u = *reinterpret_cast<const uint2*>(p + lane * 8);
          w[0] = u.x, w[1] = u.y;
        } else {
#pragma unroll
          for (int i = 0; i < W / 2; ++i) {
            const uint4 u = *reinterpret_cast<const uint4*>(p + i * 512 + lane * 16);
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
          }
        }
      };
      auto fetch = [&](int b) {
        const int j = b * 4 + n;
        if (j >= tiles.count) {  // a missing tile: zeros, under weights of zero
#pragma unroll
          for (int i = 0; i < 2 * W; ++i) kc[i] = vc[i] = 0u;
          kpar = make_uint2(0u, 0u);
          vpar = make_uint4(0u, 0u, 0u, 0u);
          return;
        }
        const uint8_t* k = kt + (size_t)tiles(j) * kv4_tile_bytes(D);
        load_codes(k, kc);
        load_codes(k + v_off, vc);
        kpar = *reinterpret_cast<const uint2*>(k + kp_off);
        vpar = *reinterpret_cast<const uint4*>(k + v_off + vp_off);
      };
      fetch(b0);
      for (int b = b0, i = it; b < b1; ++b, ++i) {
        const int s = i & 1;
        const uint32_t free_parity = (uint32_t)(((i >> 1) - 1) & 1);
        if (i >= 2 && !prompt_wait(&bars.k_empty[s], free_parity, &s_dead)) break;
        {  // slot g of the tile's first half, dimensions t D/4 + 8 w .. + 7; g + 8 of the second
          unsigned char* o = smem + C::K + s * C::KB + 2 * n * C::KS + t * W * C::KL + g * 16;
          const uint32_t s0 = __byte_perm(kpar.x, 0, 0x1010), m0 = __byte_perm(kpar.x, 0, 0x3232);
          const uint32_t s1 = __byte_perm(kpar.y, 0, 0x1010), m1 = __byte_perm(kpar.y, 0, 0x3232);
#pragma unroll
          for (int w = 0; w < W; ++w) {
            uint32_t x[4];
            dequant8(kc[w], s0, m0, x);
            *reinterpret_cast<uint4*>(o + w * C::KL) = make_uint4(x[0], x[1], x[2], x[3]);
            dequant8(kc[W + w], s1, m1, x);
            *reinterpret_cast<uint4*>(o + C::KS + w * C::KL) = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.k_full[s]);

        if (i >= 2 && !prompt_wait(&bars.v_empty[s], free_parity, &s_dead)) break;
        uint32_t bad = 0;
        const int slot0 = first_slot(b * 4 + n);
        if (!is_full(slot0) && slot0 < lim_hi) {
          // slots that no query reads become zeros, and so does a group that is not
          // finite: the queries that do read it get NaN there
          const int x = slot0 + 2 * t;
          auto live = [&](int x) { return x < lim_hi && !(x >= hole.x && x < hole.y); };
          uint32_t k0 = (live(x) ? 0xFFFFu : 0u) | (live(x + 1) ? 0xFFFF0000u : 0u);
          uint32_t k1 = (live(x + 8) ? 0xFFFFu : 0u) | (live(x + 9) ? 0xFFFF0000u : 0u);
          vpar.x &= k0, vpar.y &= k0, vpar.z &= k1, vpar.w &= k1;
          auto odd = [](uint32_t s, uint32_t m) {
            return (((s & 0x7C00u) == 0x7C00u || (m & 0x7C00u) == 0x7C00u) ? 1u : 0u) |
                   (((s & 0x7C000000u) == 0x7C000000u || (m & 0x7C000000u) == 0x7C000000u) ? 2u : 0u);
          };
          const uint32_t o0 = odd(vpar.x, vpar.y), o1 = odd(vpar.z, vpar.w);
          k0 = (o0 & 1 ? 0u : 0xFFFFu) | (o0 & 2 ? 0u : 0xFFFF0000u);
          k1 = (o1 & 1 ? 0u : 0xFFFFu) | (o1 & 2 ? 0u : 0xFFFF0000u);
          vpar.x &= k0, vpar.y &= k0, vpar.z &= k1, vpar.w &= k1;
          bad = (o0 << (2 * t)) | (o1 << (2 * t + 8));
        }
        bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
        bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
        if (t == 0) s_bad[s][n][g] = bad;
        {  // dimension g D/8 + 4 q + j of slots 2t, 2t+1 (first half of the tile), 2t+8, 2t+9 (second)
          unsigned char* o = smem + C::V + s * C::VB + 2 * n * C::VL + t * 4;
#pragma unroll
          for (int q = 0; q < W; ++q) {
            uint32_t x[4], y[4];
            dequant8(vc[q], vpar.x, vpar.y, x);
            dequant8(vc[W + q], vpar.z, vpar.w, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int d = g * (D / 8) + 4 * q + j;
              unsigned char* p = o + (d >> 3) * C::VS + (d & 7) * 16;
              *reinterpret_cast<uint32_t*>(p) = x[j];
              *reinterpret_cast<uint32_t*>(p + C::VL) = y[j];
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.v_full[s]);
        if (b + 1 < b1) fetch(b + 1);
      }
    } else if (warp == 12) {  // ---------------- issue the products
      if (lane == 0) {
        auto scores = [&](int i) {
          const int s = i & 1;
          if (!prompt_wait(&bars.k_full[s], (uint32_t)((i >> 1) & 1), &s_dead)) return false;
          tc_fence_after();
          const unsigned char* k = smem + C::K + s * C::KB;
#pragma unroll
          for (int pass = 0; pass < 2; ++pass)
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              tc_mma_f16(tmem + s * 64, smem_desc(smem + C::Q + pass * C::QB + ks * 2 * C::QL, C::QL, C::QS),
                         smem_desc(k + ks * 2 * C::KL, C::KL, C::KS), IDESC_S, (pass | ks) != 0);
          tc_commit(&bars.s_full[s]);
          tc_commit(&bars.k_empty[s]);
          return true;
        };
        bool ok = b0 < b1 && scores(it);
        for (int b = b0, i = it; b < b1 && ok; ++b, ++i) {
          const int s = i & 1;
          if (b + 1 < b1) ok = scores(i + 1);
          ok = ok && prompt_wait(&bars.v_full[s], (uint32_t)((i >> 1) & 1), &s_dead) &&
               prompt_wait(&bars.p_full, (uint32_t)(i & 1), &s_dead);
          if (!ok) break;
          tc_fence_after();
          const unsigned char* v = smem + C::V + s * C::VB;
#pragma unroll
          for (int pass = 0; pass < 2; ++pass)
#pragma unroll
            for (int ks = 0; ks < C::N / 16; ++ks)
              tc_mma_f16(tmem + C::O, smem_desc(smem + C::P + pass * C::PB + ks * 2 * C::PL, C::PL, C::PS),
                         smem_desc(v + ks * 2 * C::VL, C::VL, C::VS), IDESC_O, b > b0 || (pass | ks) != 0);
          tc_commit(&bars.pv_done);
          tc_commit(&bars.v_empty[s]);
        }
      }
    } else {  // ---------------- softmax: two threads per query
      const int half = warp >> 2, r = (warp & 3) * 32 + lane, u = u0 + r;
      const bool have = r < nq;
      const int tok = u / G;
      const size_t qi = (size_t)tok * a.q_heads + head * G + (u - tok * G);
      const int lim = have ? token_limit(a, tok, hole, false) : 0;
      const float cq = s_cq[r];
      const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      float m_ref = kNoMax, l = 0.f;
      unsigned nan_chunks = 0;  // chunks of D/8 dimensions
      bool ok = true;           // a failed wait: the warp goes on to the barriers only
      for (int b = b0, i = it; b < b1; ++b, ++i) {
        const int s = i & 1, j0 = b * 4 + 2 * half;  // this thread's tiles: j0, j0 + 1
        ok = ok && __all_sync(0xffffffffu, lane != 0 || prompt_wait(&bars.s_full[s], (uint32_t)((i >> 1) & 1), &s_dead));
        float x[32], mx = kNoMax;
        const int slot0[2] = {first_slot(j0), first_slot(j0 + 1)};
        const bool full = is_full(slot0[0]) && is_full(slot0[1]);
        if (ok) {
          tc_fence_after();
          uint32_t raw[32];
          tc_ld32(lanes + s * 64 + half * 32, raw);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(raw[j]) * cq;
          if (!full) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int p = slot0[j >> 4] + (j & 15);
              if (p >= lim || (p >= hole.x && p < hole.y)) x[j] = -INFINITY;
            }
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) mx = fmaxf(mx, x[j]);
          if (a.scores && have) {
            float* so = a.scores + qi * a.tiles * kKv4Slots;
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              if (j0 + (j >> 4) < tiles.count)
                *reinterpret_cast<float4*>(so + slot0[j >> 4] + (j & 15)) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
          }
        }
        s_pair[i & 1][half][r] = mx;
        softmax_sync();
        mx = fmaxf(mx, s_pair[i & 1][half ^ 1][r]);
        const bool raise = mx > m_ref + 8.f;
        const float corr = raise ? ex2(m_ref - mx) : 1.f;
        if (raise) {
          m_ref = mx;
          l *= corr;
        }
        // the products that read the last weights and wrote O are done
        if (i > 0)
          ok = ok && __all_sync(0xffffffffu, lane != 0 || prompt_wait(&bars.pv_done, (uint32_t)((i - 1) & 1), &s_dead));
        if (!ok) continue;
        tc_fence_after();
        if (b > b0 && __any_sync(0xffffffffu, raise)) {  // O: the thread's pair takes every other 32 columns
#pragma unroll 1
          for (int c = half * 32; c < D; c += 64) {
            uint32_t o[32];
            tc_ld32(lanes + C::O + c, o);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * corr);
            tc_st32(lanes + C::O + c, o);
          }
          tc_wait_st();
        }
        unsigned char* po = smem + C::P + (r >> 3) * C::PS + (r & 7) * 16 + half * 4 * C::PL;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t h[4], e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float v0 = ex2(x[j + 2 * k] - m_ref), v1 = ex2(x[j + 2 * k + 1] - m_ref);
            sum += v0 + v1;
            h[k] = pack2(v0, v1);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
            e[k] = pack2(v0 - f.x, v1 - f.y);
          }
          *reinterpret_cast<uint4*>(po + (j >> 3) * C::PL) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(po + C::PB + (j >> 3) * C::PL) = make_uint4(e[0], e[1], e[2], e[3]);
        }
        l += sum;
        if (!full) {  // groups that are not finite, once the block's values (and s_bad) are written
          ok = __all_sync(0xffffffffu, lane != 0 || prompt_wait(&bars.v_full[s], (uint32_t)((i >> 1) & 1), &s_dead));
          if (!ok) continue;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int c = min(max(lim - slot0[n], 0), 16);  // the query reads the tile's first c slots
            const unsigned read = (1u << c) - 1u;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (s_bad[s][2 * half + n][k] & read) nan_chunks |= 1u << k;
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full);
      }
      // ---- the item's end: the pair's sums together, every other 32 columns each
      const int n_it = b1 - b0;
      ok = ok && __all_sync(0xffffffffu, lane != 0 || prompt_wait(&bars.pv_done, (uint32_t)((it + n_it - 1) & 1), &s_dead));
      softmax_sync();  // the last maxima are read
      s_pair[0][half][r] = l;
      s_pair[1][half][r] = __uint_as_float(nan_chunks);
      softmax_sync();
      l = s_pair[0][0][r] + s_pair[0][1][r];
      nan_chunks |= __float_as_uint(s_pair[1][half ^ 1][r]);
      tc_fence_after();
      if (ok) {
        const float sink = whole && a.sink ? a.sink[head] * 1.4426950408889634f : -INFINITY;
        const float Mx = fmaxf(m_ref, sink), f = ex2(m_ref - Mx);
        const float L = l * f + (whole && a.sink ? ex2(sink - Mx) : 0.f);
        const float inv = L == 0.f ? 0.f : 1.f / L, c = whole ? f * inv : 1.f;
        float* part = a.parts + (((size_t)blockIdx.x * 2 + inside) * 128 + r) * (D + kAttn4PartHead);
        if (have && half == 0) {
          if (!whole)
            *reinterpret_cast<float2*>(part) = make_float2(m_ref, l);
          else if (a.lse)
            a.lse[qi] = make_float2(Mx, inv);
        }
#pragma unroll 1
        for (int d0 = half * 32; d0 < D; d0 += 64) {
          uint32_t o[32];
          tc_ld32(lanes + C::O + d0, o);
          tc_wait_ld();
          if (!have) continue;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float v = __uint_as_float(o[j]) * c;
            if (nan_chunks >> ((d0 + j) / (D / 8)) & 1u) v = __int_as_float(0x7FFFFFFF);
            o[j] = __float_as_uint(v);
          }
          if (whole) {
            store32(a.out, a.out_dtype, a.out_wide, (long long)qi * D + d0, o);
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4*>(part + kAttn4PartHead + d0 + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          }
        }
      }
      tc_fence_before();
    }
    it += b1 - b0;
    __syncthreads();
    tc_fence_after();
    if (s_dead) break;
    if (++head == a.nh) {
      head = 0;
      ++z;
    }
  }
  // no product may still be running when the tensor memory is freed
  if (warp == 12) {
    if (lane == 0) {
      tc_commit(&bars.all_done);
      if (!mbar_wait(&bars.all_done, 0)) s_dead = 1;
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
    if (lane == 0 && s_dead) atomicOr(a.status, kStatusTimeout);
  }
}

// Merge the partials of items that several runs share: a warp per query.
__global__ void __launch_bounds__(256) k_kv4_prompt_merge(const Kv4AttnArgs a, int n_queries, int n_z) {
  __shared__ int s_cum[kPromptMaxZ + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = a.D, G = a.q_heads / a.nh;
  const int z = blockIdx.x / a.nh, head = blockIdx.x % a.nh;
  Attn4Runs runs;
  prompt_runs(a, n_queries, n_z, s_cum, runs);  // positions and holes: written before the attention began
  pdl_launch_dependents();
  const int s = runs.start(z, head) + kPromptStart, cnt = runs.tiles(z) - kPromptStart;
  const int c0 = s / runs.per, n = cnt ? (s + cnt - 1) / runs.per - c0 + 1 : 0;
  pdl_wait();
  if (n <= 1) return;  // one run's: finished there
  const float sink = a.sink ? a.sink[head] * 1.4426950408889634f : -INFINITY;
  const size_t step = (size_t)2 * 128 * (D + kAttn4PartHead);
  // a run's second partial is of an item that begins inside it: the first run's, if any
  const size_t shift = s > c0 * runs.per ? step / 2 : 0;
  for (int r = blockIdx.y * 16 + warp; r < blockIdx.y * 16 + 16; r += 8) {
    const int u = z * 128 + r;
    if (u >= n_queries) break;
    const float* base = a.parts + c0 * step + (size_t)r * (D + kAttn4PartHead);
    auto part = [&](int c) { return base + c * step + (c ? 0 : shift); };
    float m = kNoMax, l = 0.f;
    for (int c = lane; c < n; c += 32) {
      const float2 p = *reinterpret_cast<const float2*>(part(c));
      const float hi = fmaxf(m, p.x);
      l = l * ex2(m - hi) + p.y * ex2(p.x - hi);
      m = hi;
    }
    float M = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    M = fmaxf(M, sink);
    float L = l * ex2(m - M);
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (a.sink) L += ex2(sink - M);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int c = 0; c < n; ++c) {
      const float* p = part(c);
      const float f = ex2(p[0] - M);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (32 * k < D) v[k] += p[kAttn4PartHead + lane + 32 * k] * f;
    }
    const int tok = u / G;
    const long long qi = (long long)tok * a.q_heads + head * G + (u - tok * G);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (32 * k < D) store_elem(a.out, a.out_dtype, qi * D + lane + 32 * k, v[k] * inv);
    if (a.lse && lane == 0) a.lse[qi] = make_float2(M, inv);
  }
}

template <int D>
static cudaError_t launch_prompt4(const Kv4AttnArgs& args, int tokens, cudaStream_t st, bool pdl) {
  Kv4AttnArgs a = args;
  a.q_wide = (uintptr_t)a.q % 16 == 0;
  a.out_wide = (uintptr_t)a.out % 16 == 0;
  const int queries = tokens * (a.q_heads / a.nh), n_z = (queries + 127) / 128;
  const long long items = (long long)n_z * a.nh;
  // one run per SM, unless there are so many items that their last wave does not show
  const int ctas = a.n_sm * 256 <= kAttn4MaxParts * 2 ? a.n_sm : kAttn4MaxParts * 2 / 256;
  a.n_runs = items >= 8LL * ctas || n_z > kPromptMaxZ ? 0 : ctas;
  cudaError_t e = launch_kernel(k_kv4_prompt<D>, dim3(a.n_runs ? a.n_runs : (unsigned)items), dim3(kPromptThreads),
                                (size_t)Prompt4<D>::SMEM, st, pdl, a, queries, n_z);
  if (e == cudaSuccess && a.n_runs)
    e = launch_kernel(k_kv4_prompt_merge, dim3((unsigned)items, 8), dim3(256), 0, st, true, a, queries, n_z);
  return e;
}

cudaError_t launch_kv4_prompt(const Kv4AttnArgs& a, int tokens, cudaStream_t st, bool pdl) {
  switch (a.D) {
    case 32: return launch_prompt4<32>(a, tokens, st, pdl);
    case 64: return launch_prompt4<64>(a, tokens, st, pdl);
    case 128: return launch_prompt4<128>(a, tokens, st, pdl);
  }
  return cudaErrorInvalidValue;
}

cudaError_t init_kv4_prompt_attributes() {
  cudaError_t e = allow_max_dyn_smem(k_kv4_prompt<32>);
  if (e == cudaSuccess) e = allow_max_dyn_smem(k_kv4_prompt<64>);
  if (e == cudaSuccess) e = allow_max_dyn_smem(k_kv4_prompt<128>);
  return e;
}

}  // namespace uocr
