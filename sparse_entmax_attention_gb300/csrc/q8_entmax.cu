// q8_entmax.cu -- alpha-entmax decode over the 8-bit paged cache, one new token
// a sequence.
//
//   z_j = (α−1)·s_j,  Σ_j [z_j − τ]_+^β = 1 (β = 1/(α−1)),  o = Σ_j [z_j − τ]_+^β v_j.
//
// 1. score: K streams once, on the same line of 32-key tiles as the softmax
//    kernel; z and each tile's largest z go to the workspace. Bound: K's bytes.
// 2. finish: a cluster of eight blocks per (slot, KV head), each with an eighth
//    of the tiles. No token at or below z_max − 1 can carry weight (τ ≥ z_max − 1,
//    where the sum is at least 1), so only tiles whose largest z clears that are
//    looked at again: their scores go to every block of the cluster, and each
//    solves alone, from z_max − 1 until the weights' sum is 1 (EntSolve). (Where
//    there are too many scores to hand round, a step's partial sums are instead,
//    with a cluster barrier each.)
//    Then V is read for tiles with some z above its head's τ only, weights
//    rounded to halves against their tile's largest (off by 2^-11, an eighth of the
//    bf16 output's rounding), and the blocks' sums are
//    added through the cluster. Every sum has a fixed order.
//
// Measured, 8 KV heads of 4 query heads, d = 128: 131072 tokens, int8, slopes,
// alpha 1.5: 56.6 us, of which scoring is 33 (134 MB of K at 4.1 TB/s; the floor is
// 20): turning codes into halves bounds it (ALU 49%, IPC 2.3, DRAM 53%), 16 and
// 24 warps alike. The rest is a chain of short phases, most of each the fetch of
// its instructions. 16 sequences of 1-32k tokens, e4m3, alpha 2: 64 us. Dense
// supports (random scores of deviation 1, 131072 tokens, every step reads z
// again): 103 us at alpha 1.5, 152 at 1.25; equal scores 140 and 132 (110 and 128
// without the step that shows the sum to be 1).
#include "q8_tiles.cuh"

namespace ekv {

constexpr int kScoreWarps = 24;
constexpr int kScoreSlabs = 2;
constexpr int kEntWarps = 16;
constexpr int kEntKeys = 32;
constexpr int kEntCluster = 8;  // blocks of a cluster, at most
constexpr int kEntSent = 64;  // scores a warp hands round the cluster, at most
constexpr int kEntList = kEntWarps * 32;  // tiles listed at once

struct EntArgs {
  Q8AttendArgs a;
  float a1, beta;
  float* z;     // [tile of the line][G][32]
  float* pmax;  // [tile of the line][G]
  struct EntUnit* slots;  // [n_seqs]
};
// What the scoring kernel leaves of a slot for the finishing one.
struct __align__(16) EntUnit {
  Q8Slot s;
  Q8Span sp;
  int T, pad[2];
  long long cum;
};

__device__ __forceinline__ Q8Span ent_span(const Q8AttendArgs& a, const Q8Slot& s, int b) {
  return q8_span(a.c, a.sc, s, b, 0, 1);
}
__device__ __forceinline__ int ent_tiles(const Q8Span& sp, int P) { return (sp.T * P + kEntKeys - 1) / kEntKeys; }

template <bool I8, int D, int P>
__global__ void __launch_bounds__(kScoreWarps * 32, 1)
    ent_score_kernel(EntArgs e, const __grid_constant__ CUtensorMap kmap) {
  pdl_enter();
  constexpr int NW = kScoreWarps, ST = kScoreSlabs, SLAB = kEntKeys * D, PP = kEntKeys / P;
  extern __shared__ __align__(128) unsigned char dyn_sm[];
  __shared__ uint64_t bars[NW][ST];
  __shared__ LineSmem<NW> sh_line;
  const Q8AttendArgs& a = e.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = ((smem_u32(dyn_sm) + 1023u) & ~1023u) + (uint32_t)warp * ST * SLAB;
  unsigned char* ring_p = dyn_sm + (ring - smem_u32(dyn_sm));
  if (lane == 0) {
    for (int i = 0; i < ST; ++i) mbar_init(&bars[warp][i], 1);
    mbar_fence_init();
  }
  const int Hkv = a.c.Hkv, G = a.c.G;
  if (tid == 0) prefetch_map(&kmap);
  const LinePlace at = line_place<NW>(
      a.b.n_seqs, a.c.status, sh_line,
      [&](int b, uint32_t* st) {
        const Q8Slot s = q8_slot(a.c, a.b, b, st);
        return s.count > 0 ? (long long)ent_tiles(ent_span(a, s, b), P) * Hkv : 0LL;
      },
      [&](int b, long long where) {
        if (b >= a.b.n_seqs) return;
        EntUnit u;
        u.s = q8_slot(a.c, a.b, b, nullptr);
        u.sp = u.s.count > 0 ? ent_span(a, u.s, b) : Q8Span{0, 0, 0, 0, 0};
        u.T = ent_tiles(u.sp, P);
        u.pad[0] = u.pad[1] = 0;
        u.cum = where;
        e.slots[b] = u;
      });
  const long long w_end = at.end;
  if (at.begin >= w_end) return;
  const int r = lane >> 2, c = lane & 3;
  int slot = at.slot;
  long long cum = at.cum, w = at.begin;
  int filled = 0, used = 0;
  bool stuck = false;
  while (w < w_end && !stuck) {
    const Q8Slot s = q8_slot(a.c, a.b, slot, nullptr);
    const Q8Span sp = s.count > 0 ? ent_span(a, s, slot) : Q8Span{0, 0, 0, 0, 0};
    const int T = ent_tiles(sp, P);
    if (w >= cum + (long long)T * Hkv) {
      cum += (long long)T * Hkv;
      ++slot;
      continue;
    }
    const long long off = w - cum;
    const int kvh = (int)div_line(off, T), t0 = (int)(off - (long long)kvh * T);
    const int n = (int)min((long long)(T - t0), w_end - w);
    uint4 qw[D / 32];
    q_load<D>(r < G ? a.q.p + (long long)s.start * a.q.ts + (long long)(kvh * G + r) * a.q.hs : nullptr, lane, qw);
    const int pos = s.L - 1;
    int lo = a.sc.window > 0 ? max(0, pos - a.sc.window + 1) : 0;
    if (a.sc.first_key) lo = max(lo, a.sc.first_key[s.start]);
    // 32 tiles' places and scales at once, a tile a lane; bits of those with a page, and of those seen whole
    int ph[PP], key_l[PP];
    float ks_l[PP];
    uint32_t some_bits = 0u, whole_bits = 0u;
    auto look_up = [&](int p0) {
      bool some = false, whole = true;
#pragma unroll
      for (int q = 0; q < PP; ++q) {
        const int t = (t0 + p0 + lane) * PP + q;
        ph[q] = -1;
        ks_l[q] = 0.0f;
        key_l[q] = kNoKey;
        if (p0 + lane < n && t < sp.T) {
          const int page = sp.page(t);
          ph[q] = phys_page(a.c.block_table, s.seq, page, a.c.maxp, a.c.nphys, a.c.status);
          if (ph[q] >= 0) {
            ks_l[q] = a.c.k_scale[(size_t)ph[q] * Hkv + kvh];
            key_l[q] = page * P;
            some = true;
          }
        }
        whole &= (key_l[q] + P - 1 <= pos && key_l[q] >= lo) || key_l[q] + P <= sp.pre;
      }
      some_bits = __ballot_sync(0xffffffffu, some);
      whole_bits = __ballot_sync(0xffffffffu, whole);
    };
    int ask = 0;
    auto refill = [&](int end) {
      while (ask < end && filled - used < ST) {
        if (some_bits >> (ask & 31) & 1u) {
          int f[PP], there = 0;
#pragma unroll
          for (int q = 0; q < PP; ++q) {
            f[q] = __shfl_sync(0xffffffffu, ph[q], ask & 31);
            there += f[q] >= 0;
          }
          const int sg = filled % ST;
          if (lane == 0) {
            mbar_expect_tx(&bars[warp][sg], (uint32_t)(there * P * D));
#pragma unroll
            for (int q = 0; q < PP; ++q)
              if (f[q] >= 0) tma_load_3d(ring_p + sg * SLAB + q * P * D, &kmap, 0, kvh * P, f[q], &bars[warp][sg]);
          }
          ++filled;
        }
        ++ask;
      }
    };
    look_up(0);
    refill(min(n, 32));
    uint32_t bq[1][D / 16][2];
    Q8Row row[2];
    float inv;
    q_half_frag<D>(qw, bq[0], inv);
    const bool mine[2] = {2 * c < G, 2 * c + 1 < G};
    float* zo = e.z + ((size_t)w * G + 2 * c) * kEntKeys + r;  // this lane's scores of the tile
    float* po = e.pmax + (size_t)w * G + 2 * c;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      row[j].cs = q8_row_scale(__shfl_sync(0xffffffffu, inv, (2 * c + j) * 4), a.sc, e.a1);
      row[j].slope = a.sc.slopes && 2 * c + j < G ? a.sc.slopes[kvh * G + 2 * c + j] * e.a1 : 0.0f;
      row[j].pos = pos;
      row[j].lo = lo;
    }
    for (int i = 0; i < n; ++i) {
      if ((i & 31) == 0 && i) {
        look_up(i);
        refill(min(n, i + 32));
      }
      const bool some = some_bits >> (i & 31) & 1u, whole = whole_bits >> (i & 31) & 1u;
      if (some && !__all_sync(0xffffffffu, mbar_wait_bounded(&bars[warp][used % ST], (used / ST) & 1))) {
        stuck = true;
        break;
      }
      const uint32_t slab = ring + (used % ST) * SLAB;
      float pm[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        constexpr int kHalf = 16;
        const int q = kHalf * mt / P;
        const float ks = __shfl_sync(0xffffffffu, ks_l[q], i & 31);
        const int j0 = __shfl_sync(0xffffffffu, key_l[q], i & 31) + (kHalf * mt) % P + r;
        float acc[1][4] = {{0.f, 0.f, 0.f, 0.f}};
        if (some) k_dot<I8, D, 1>(slab, kHalf * mt, lane, bq, acc);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float dot[2] = {acc[0][j], acc[0][2 + j]};
          float v[2];
          q8_scores(dot, v, row[j], ks, j0, a.sc, e.a1, 0.0f);
          if (!whole) {
            if (!q8_sees(row[j], j0, sp.pre)) v[0] = -CUDART_INF_F;
            if (!q8_sees(row[j], j0 + 8, sp.pre)) v[1] = -CUDART_INF_F;
          }
          if (mine[j]) {
            zo[j * kEntKeys + kHalf * mt] = v[0];
            zo[j * kEntKeys + kHalf * mt + 8] = v[1];
          }
          pm[j] = max3_nan(pm[j], v[0], v[1]);
        }
      }
      zo += G * kEntKeys;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        pm[j] = max_nan(pm[j], __shfl_xor_sync(0xffffffffu, pm[j], 4));
        pm[j] = max_nan(pm[j], __shfl_xor_sync(0xffffffffu, pm[j], 8));
        pm[j] = max_nan(pm[j], __shfl_xor_sync(0xffffffffu, pm[j], 16));
        if (r == 0 && mine[j]) po[j] = pm[j];
      }
      po += G;
      if (some) {
        __syncwarp();
        ++used;
        refill(min(n, (i | 31) + 1));
      }
    }
    w += n;
  }
  if (stuck) {
    if (lane == 0) {
      raise_flag(a.c.status, ENTMAXKV_DEV_TIMEOUT);
      for (; used < filled; ++used) mbar_wait_bounded(&bars[warp][used % ST], (used / ST) & 1);
    }
    __syncwarp();
  }
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// The address of a shared object in another block of the cluster.
__device__ __forceinline__ uint32_t peer(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void peer_store4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ float peer_load(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// x^b for x ≥ 2^-126 at an order without a short form, as 2^{b·lg x}: the
// logarithm is good to 2^-22 of itself (or absolutely, near 1), so a power is to
// b·|lg x|·2^-22 and x^b times that to 2^-22.
__device__ __forceinline__ float lg2f(float x) {
  float l;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(l) : "f"(x));
  return l;
}
__device__ __forceinline__ float ent_pow(float x, float b) { return ex2f(b * lg2f(x)); }
constexpr float kLeast = 0x1p-126f;  // a smaller z − τ carries no weight
__device__ __forceinline__ float ent_weight(float y, float beta) {  // [y]_+^β
  y = fmaxf(y, 0.0f);
  if (beta == 2.0f) return y * y;
  if (beta == 1.0f) return y;
  return y >= kLeast ? ent_pow(y, beta) : 0.0f;
}

// A head's threshold: τ = top + a + b, top its largest score. The two parts of
// τ − top keep a difference of any size: b's own 24 bits hold y where a is the
// score that is left (a y of 1e-10 beside an offset of 0.3 has its weight's share
// at an order above 2, and equal scores share it).
struct EntTau {
  float top, a, b;
  __device__ __forceinline__ float over(float z) const { return ((z - top) - a) - b; }
};

// What one step of the solve learns of the scores' offsets d = z − top with
// y = d − (a + b) > 0: their number, Σy and Σy² (Σy^{β−1} and Σy^β for other
// orders), and the least of the offsets.
struct EntSums {
  float k, s1, s2, least;
  __device__ __forceinline__ void add(float d, float y, float beta, bool low) {
    if (y >= kLeast) {
      k += 1.0f;
      least = fminf(least, d);
      const float w = low ? y : ent_pow(y, beta - 1.0f);
      s1 += w;
      s2 = fmaf(w, y, s2);
    }
  }
  __device__ __forceinline__ void warp_total() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      k += __shfl_xor_sync(0xffffffffu, k, o);
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
    }
  }
};
// s += x with what the additions before lost: a lane's sum over a million tiles keeps its 24 bits.
__device__ __forceinline__ void add_kept(float& s, float& lost, float x) {
  const float y = x - lost, t = s + y;
  lost = (t - s) - y;
  s = t;
}

// A number of 48 bits, h + l with l within half of h's last bit.
struct Pair {
  float h, l;
  __device__ __forceinline__ Pair plus(float x) const {
    const float s = h + x, v = s - h, r = ((h - (s - v)) + (x - v)) + l;
    const float t = s + r;
    return Pair{t, r - (t - s)};
  }
  __device__ __forceinline__ float minus(const Pair& o) const { return (h - o.h) + (l - o.l); }
};

// The threshold of one head, as the offset t = τ − top in [−1, 0), moved by the
// sums of a step until the weights' sum S is 1: to kNear + β·2^-21, which is the
// powers' own error (and to a 64th of that where the steps still gain). Steps:
//   β = 2, 1  the closed-form root where it keeps the support, which ends the
//             solve from S ≤ 1.25 (from farther off its rounding shows, and it is
//             a step like others), else
//   Newton on the norm S^{1/β} (β = 1: on S), convex and falling for β ≥ 1, so
//             that steps from S ≥ 1 stay below the root and nearly reach it on
//             equal scores; close to 1 on S itself.
// For β < 1 the sum's slope has no bound where a score enters, so every step lies
// in a bracket, and one that leaves it, or does not halve |S − 1|, becomes the
// bracket's middle (in the logarithm where its ends are far apart: n equal scores
// have t = −n^{−1/β}). A bracket that closes on a score is continued in distances
// from that score.
constexpr int kEntSteps = 100;
struct EntSolve {
  static constexpr float kNear = 0x1p-14f, kFirst = 0x1p127f;
  Pair t, lo, hi;     // from `org`; S(lo) ≥ 1 > S(hi)
  float org, a, b;    // a + b = org + t
  float prev, at_lo;  // |S − 1| of the step before, the least offset of the support at lo
  bool done;
  __device__ __forceinline__ explicit EntSolve(bool skip)
      : t{-1.0f, 0.0f}, lo{-1.0f, 0.0f}, hi{0.0f, 0.0f}, org(0.0f), a(-1.0f), b(0.0f), prev(kFirst), at_lo(0.0f), done(skip) {}
  __device__ __forceinline__ float over(float d) const { return (d - a) - b; }
  __device__ __forceinline__ void step(const EntSums& v, float beta) {
    const bool two = beta == 2.0f, one = beta == 1.0f;
    const float S = one ? v.s1 : v.s2, slope = one ? v.k : v.s1;  // slope · β is the sum's
    const float e = S - 1.0f, ae = fabsf(e), inv = 1.0f / beta;
    const float near = kNear + beta * 0x1p-21f;
    if (e < 0.0f) {
      hi = t;
    } else {
      lo = t;
      at_lo = v.least;
    }
    // no root above −k^{−1/β}, k scores at −1 (1/64: the powers' error)
    if (prev == kFirst && beta < 1.0f) hi = Pair{-0.984375f * ent_pow(v.k, -inv), 0.0f};
    if (ae <= 0x1p-6f * near || (ae <= near && ae > 0.5f * prev)) {
      done = true;
      return;
    }
    float st = __fdividef(e, beta * slope);
    bool last = beta >= 1.0f && e > 0.0f && ae <= near;
    if (two || one) {
      const float disc = slope * slope - v.k * e;  // Σ(y − δ)² = 1, without cancellation
      const float d = one ? st : disc >= 0.0f ? __fdividef(e, slope + sqrtf(disc)) : CUDART_INF_F;
      if (d <= (v.least - a) - b) {
        st = d;
        last = e > 0.0f && ae <= 0.25f;
      } else if (two && e > 0.0f && !last) {
        st = __fdividef(S - sqrtf(S), slope);
      }
    } else if (!last && (beta < 1.0f || S > 1.5f)) {
      st = __fdividef(S - ent_pow(S, 1.0f - inv), slope);
    }
    if (last) {
      b += st;
      done = true;
      return;
    }
    Pair to = t.plus(st);
    if (!(to.minus(lo) > 0.0f && to.minus(hi) < 0.0f) || ae > 0.5f * prev) {
      if (org == 0.0f && hi.minus(lo) <= -0x1p-40f * lo.h) {
        org = at_lo;
        lo = Pair{fminf(lo.minus(Pair{org, 0.0f}), -0x1p-119f), 0.0f};
        hi = Pair{fminf(hi.minus(Pair{org, 0.0f}), -0x1p-120f), 0.0f};
      }
      to = beta < 1.0f && lo.h < 4.0f * hi.h ? Pair{-ex2f(0.5f * (lg2f(-lo.h) + lg2f(-hi.h))), 0.0f}
                                             : lo.plus(0.5f * hi.minus(lo));
    }
    prev = ae;
    t = to;
    a = org == 0.0f ? t.h : org;
    b = org == 0.0f ? t.l : t.h;
  }
};

template <bool I8, int D, int P>
__global__ void __launch_bounds__(kEntWarps * 32, 1)
    ent_finish_kernel(EntArgs e, const __grid_constant__ CUtensorMap vmap) {
  pdl_enter();
  constexpr int NW = kEntWarps, SLAB = kEntKeys * D, PP = kEntKeys / P, NTH = NW * 32;
  extern __shared__ __align__(128) unsigned char dyn_sm[];
  __shared__ uint64_t bars[NW][2];
  __shared__ float4 sums[2][kEntCluster][NW];  // every warp of the cluster's partial sums, two steps in turn
  __shared__ int counts[kEntCluster][NW];      // scores a warp has handed round; over kEntSent: too many
  __shared__ float top_sh[kEntCluster][8];
  __shared__ float wtop[NW][8];
  __shared__ EntTau tau_sh[8];
  __shared__ int found[NW + 1];
  __shared__ __align__(16) float part[8 * D];
  const Q8AttendArgs& a = e.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = gridDim.x;  // the cluster
  const int rank = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z, G = a.c.G, Hkv = a.c.Hkv;
  const uint32_t base = (smem_u32(dyn_sm) + 1023u) & ~1023u;
  unsigned char* base_p = dyn_sm + (base - smem_u32(dyn_sm));
  if (lane == 0) {
    mbar_init(&bars[warp][0], 1);
    mbar_init(&bars[warp][1], 1);
    mbar_fence_init();
  }
  if (tid == 0) prefetch_map(&vmap);
  const EntUnit unit = e.slots[b];
  const Q8Slot s = unit.s;
  if (s.count == 0) return;  // (the whole cluster)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
  const Q8Span sp = unit.sp;
  const int T = unit.T;
  const size_t tile0 = (size_t)(unit.cum + (long long)kvh * T);
  const int lo = (int)((long long)T * rank / C), hi = (int)((long long)T * (rank + 1) / C);
  const float* pmax = e.pmax + tile0 * G;

  // each head's largest score
  {
    float m[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) m[h] = -CUDART_INF_F;
    for (int t = lo + tid; t < hi; t += NTH)
#pragma unroll
      for (int h = 0; h < 8; ++h)
        if (h < G) m[h] = max_nan(m[h], pmax[(size_t)t * G + h]);
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      if (h < G)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m[h] = max_nan(m[h], __shfl_xor_sync(0xffffffffu, m[h], o));
      if (lane == 0) wtop[warp][h] = m[h];
    }
    __syncthreads();
    // every block of the cluster is running before the first store into another's shared memory
    asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    if (tid < 8 * C) {
      const int h = tid & 7;
      float v = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < NW; ++i) v = max_nan(v, wtop[i][h]);
      asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(peer(smem_u32(&top_sh[rank][h]), tid >> 3)), "f"(v)
                   : "memory");
    }
    cluster_sync();
  }
  // The block's warps share out the heads, a head's warps its part of the tiles. Scores above z_max − 1 go to every
  // block of the cluster as offsets from z_max, kEntSent a warp at most, so that each can solve alone.
  const int wph = NW / G, hd = warp / wph, wi = warp % wph;
  const bool works = hd < G;
  float top = -CUDART_INF_F;
  if (works)
    for (int i = 0; i < C; ++i) top = max_nan(top, top_sh[i][hd]);
  // a head without keys answers 0; one with a score that is NaN or +∞ answers NaN, as its b says
  const bool odd = !(top < CUDART_INF_F), none = odd || top == -CUDART_INF_F;
  const int wlo = lo + (int)((long long)(hi - lo) * wi / wph), whi = lo + (int)((long long)(hi - lo) * (wi + 1) / wph);
  float* sent = reinterpret_cast<float*>(base_p);                     // [cluster][warps][kEntSent] offsets from top
  const float* zh = e.z + (tile0 * G + (works ? hd : 0)) * kEntKeys;  // tile t's scores at zh + t·G·32
  int n_sent = 0;
  if (works && !none) {
    for (int t1 = wlo; t1 < whi && n_sent <= kEntSent; t1 += 128) {
      float m[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        m[k] = t1 + 32 * k + lane < whi ? pmax[(size_t)(t1 + 32 * k + lane) * G + hd] : -CUDART_INF_F;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t in = __ballot_sync(0xffffffffu, m[k] - top > -1.0f);
        while (in && n_sent <= kEntSent) {  // four tiles' scores in flight
          float z[4];
          const int n4 = min(4, __popc(in));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            z[i] = i < n4 ? zh[(size_t)(t1 + 32 * k + __ffs(in) - 1) * G * kEntKeys + lane] : -CUDART_INF_F;
            in &= in - 1u;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float d = z[i] - top;
            const uint32_t up = __ballot_sync(0xffffffffu, d > -1.0f);
            const int at = n_sent + __popc(up & ((1u << lane) - 1u));
            if (d > -1.0f && at < kEntSent)
              for (int k2 = 0; k2 < C; ++k2)
                asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(
                                 peer(smem_u32(&sent[(rank * NW + warp) * kEntSent + at]), k2)),
                             "f"(d)
                             : "memory");
            n_sent += __popc(up);
          }
        }
      }
    }
  }
  if (lane < C)
    asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(peer(smem_u32(&counts[rank][warp]), lane)), "r"(n_sent)
                 : "memory");
  cluster_sync();
  bool many = false;  // some warp had more: the sums of a step are exchanged instead
  for (int i = lane; i < C * NW; i += 32) many |= counts[i / NW][i % NW] > kEntSent;
  many = __any_sync(0xffffffffu, many);
  const bool low = e.beta == 2.0f || e.beta == 1.0f;
  EntSolve sv(!works || none);
  if (!many) {
    if (wi == 0) {  // a head's first warp, a lane or more a segment
      for (int it = 0; it < kEntSteps && !sv.done; ++it) {
        EntSums v{0.0f, 0.0f, 0.0f, CUDART_INF_F};
        for (int i = lane; i < C * wph; i += 32) {
          const int g = (i / wph) * NW + hd * wph + i % wph;
          const int n = counts[g / NW][g % NW];
          for (int k = 0; k < n; ++k) {
            const float d = sent[g * kEntSent + k];
            v.add(d, sv.over(d), e.beta, low);
          }
        }
        v.warp_total();
        sv.step(v, e.beta);
      }
    }
  } else {
    for (int it = 0; it < kEntSteps; ++it) {
      EntSums v{0.0f, 0.0f, 0.0f, CUDART_INF_F};
      if (!sv.done) {
        float lost1 = 0.0f, lost2 = 0.0f;
        for (int t1 = wlo; t1 < whi; t1 += 32) {
          uint32_t in = __ballot_sync(0xffffffffu, t1 + lane < whi && sv.over(pmax[(size_t)(t1 + lane) * G + hd] - top) > 0.0f);
          while (in) {  // eight tiles' scores in flight
            float z[8];
            const int n8 = min(8, __popc(in));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              z[i] = i < n8 ? zh[(size_t)(t1 + __ffs(in) - 1) * G * kEntKeys + lane] : -CUDART_INF_F;
              in &= in - 1u;
            }
            EntSums u{0.0f, 0.0f, 0.0f, CUDART_INF_F};
#pragma unroll
            for (int i = 0; i < 8; ++i) u.add(z[i] - top, sv.over(z[i] - top), e.beta, low);
            v.k += u.k;
            v.least = fminf(v.least, u.least);
            add_kept(v.s1, lost1, u.s1);
            add_kept(v.s2, lost2, u.s2);
          }
        }
        v.warp_total();
      }
      if (lane < C)
        peer_store4(peer(smem_u32(&sums[it & 1][rank][warp]), lane),
                    make_float4(sv.done ? -1.0f : v.k, v.s1, v.s2, v.least));
      cluster_sync();
      // every head done? (its first warp in the first block says so)
      const bool hd_done = lane >= G || sums[it & 1][0][lane * wph].x < 0.0f;
      if (__all_sync(0xffffffffu, hd_done)) break;
      if (sv.done) continue;
      v = EntSums{0.0f, 0.0f, 0.0f, CUDART_INF_F};
      for (int i = lane; i < C * wph; i += 32) {
        const float4 p = sums[it & 1][i / wph][hd * wph + i % wph];
        v.k += p.x;
        v.s1 += p.y;
        v.s2 += p.z;
        v.least = fminf(v.least, p.w);
      }
      v.warp_total();
      sv.step(v, e.beta);
    }
  }
  if (works && wi == 0 && lane == 0) {
    tau_sh[hd] = EntTau{none ? CUDART_NAN_F : top, sv.a, odd ? CUDART_NAN_F : sv.b};
    if (rank == 0) {
      if (!sv.done) raise_flag(a.c.status, ENTMAXKV_DEV_TAU_NOCONV);
      if (a.tau) a.tau[(size_t)s.start * Hkv * G + kvh * G + hd] = none ? CUDART_NAN_F : top + (sv.a + sv.b);
    }
  }
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");  // the copies below write where scores were kept
  __syncthreads();

  // Weights and V. The block's tiles with some score above its head's τ are listed in order, and its warps take them
  // in turns, the next one's V on its way.
  int* list = reinterpret_cast<int*>(base_p + 2 * NW * SLAB);  // [kEntList] tiles
  const int r = lane >> 2, c = lane & 3;
  const EntTau tau_r = r < G ? tau_sh[r] : EntTau{CUDART_INF_F, 0.0f, 0.0f};
  float acc[D / 16][1][4];
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) acc[mt][0][0] = acc[mt][0][1] = acc[mt][0][2] = acc[mt][0][3] = 0.0f;
  int used = 0;
  bool stuck = false;
  for (int l0 = lo; l0 < hi; l0 += kEntList) {
    const int t = l0 + tid;
    bool in = false;
    if (t < hi && t < l0 + kEntList)
      for (int h = 0; h < G; ++h) in |= tau_sh[h].over(pmax[(size_t)t * G + h]) > 0.0f;
    const uint32_t bits = __ballot_sync(0xffffffffu, in);
    if (lane == 0) found[warp] = __popc(bits);
    __syncthreads();
    int at = 0, all = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      if (i < warp) at += found[i];
      all += found[i];
    }
    if (in) list[at + __popc(bits & ((1u << lane) - 1u))] = t;
    __syncthreads();
    // this warp's tiles: list[warp], list[warp + NW], ...; their places, a tile a lane
    const int mine = all > warp ? (all - warp + NW - 1) / NW : 0;
    int ph[PP], tl = -1;
    float vs_l[PP];
#pragma unroll
    for (int q = 0; q < PP; ++q) {
      ph[q] = -1;
      vs_l[q] = 0.0f;
    }
    if (lane < mine) {
      tl = list[warp + lane * NW];
#pragma unroll
      for (int q = 0; q < PP; ++q) {
        const int p = tl * PP + q;
        if (p < sp.T) ph[q] = phys_page(a.c.block_table, s.seq, sp.page(p), a.c.maxp, a.c.nphys, nullptr);
        if (ph[q] >= 0) vs_l[q] = a.c.v_scale[(size_t)ph[q] * Hkv + kvh];
      }
    }
    auto ask = [&](int i) {
      int f[PP], there = 0;
#pragma unroll
      for (int q = 0; q < PP; ++q) {
        f[q] = __shfl_sync(0xffffffffu, ph[q], i);
        there += f[q] >= 0;
      }
      if (lane == 0) {  // (a tile without a page completes at once)
        uint64_t* bar = &bars[warp][(used + i) & 1];
        mbar_expect_tx(bar, (uint32_t)(there * P * D));
#pragma unroll
        for (int q = 0; q < PP; ++q)
          if (f[q] >= 0)
            tma_load_3d(base_p + (warp * 2 + ((used + i) & 1)) * SLAB + q * P * D, &vmap, 0, kvh * P, f[q], bar);
      }
    };
    if (mine > 0) ask(0);
    for (int i = 0; i < mine; ++i) {
      if (i + 1 < mine) ask(i + 1);
      const int tt = __shfl_sync(0xffffffffu, tl, i);
      int f[PP];
      float vs[PP];
#pragma unroll
      for (int q = 0; q < PP; ++q) {
        f[q] = __shfl_sync(0xffffffffu, ph[q], i);
        vs[q] = __shfl_sync(0xffffffffu, vs_l[q], i);
      }
      // row r's weights of this tile against a power of two above its largest; the V scales of a tile's two pages
      // differ: each goes into its own keys' weights, over the larger of them
      const float ym = r < G ? tau_r.over(pmax[(size_t)tt * G + r]) : -1.0f;
      float2 z[2][2];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          z[kt][j] = r < G ? *reinterpret_cast<const float2*>(e.z + ((tile0 + tt) * G + r) * kEntKeys + 16 * kt + 8 * j + 2 * c)
                           : make_float2(-CUDART_INF_F, -CUDART_INF_F);
      const float vmax = PP == 1 ? vs[0] : fmaxf(vs[0], vs[PP - 1]);
      const float vinv = vmax > 0.0f ? 1.0f / vmax : 0.0f;
      const float most = ent_weight(ym, e.beta);
      const int ex = min(max((int)(__float_as_uint(most) >> 23) - 126, -100), 100);
      const float up = __uint_as_float((uint32_t)(127 - ex) << 23), down = __uint_as_float((uint32_t)(127 + ex) << 23);
      uint32_t bf[2][1][2];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        const float f0 = PP == 1 ? up : up * (vs[16 * kt / P] * vinv);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float y0 = tau_r.over(z[kt][j].x), y1 = tau_r.over(z[kt][j].y);
          const __half2 p = __floats2half2_rn(ent_weight(y0, e.beta) * f0, ent_weight(y1, e.beta) * f0);
          bf[kt][0][j] = *reinterpret_cast<const uint32_t*>(&p);
        }
      }
      const int n = used + i, sg = n & 1;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bars[warp][sg], (uint32_t)(n >> 1) & 1u))) {
        stuck = true;
        break;
      }
      const uint32_t slab = base + (warp * 2 + sg) * SLAB;
      unsigned char* slab_p = base_p + (warp * 2 + sg) * SLAB;
      bool wrote = false;  // places past the sequence's end, or of no page: any bytes, so that w = 0 meets no NaN
#pragma unroll
      for (int q = 0; q < PP; ++q) {
        const int nv = f[q] >= 0 ? min(P, s.L - sp.page(tt * PP + q) * P) : 0;
        if (nv == P) continue;
        for (int k = lane; k < (P - nv) * (D / 16); k += 32)
          *reinterpret_cast<uint4*>(slab_p + (q * P + nv) * D + k * 16) = make_uint4(0u, 0u, 0u, 0u);
        wrote = true;
      }
      if (wrote) {
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
      }
      float tmp[D / 16][1][4];
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) tmp[mt][0][0] = tmp[mt][0][1] = tmp[mt][0][2] = tmp[mt][0][3] = 0.0f;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) v_dot<I8, D, 1>(slab, 16 * kt, lane, bf[kt], tmp);
      const float f0 = __shfl_sync(0xffffffffu, down, 8 * c) * vmax, f1 = __shfl_sync(0xffffffffu, down, 8 * c + 4) * vmax;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        acc[mt][0][0] = fmaf(tmp[mt][0][0], f0, acc[mt][0][0]);
        acc[mt][0][2] = fmaf(tmp[mt][0][2], f0, acc[mt][0][2]);
        acc[mt][0][1] = fmaf(tmp[mt][0][1], f1, acc[mt][0][1]);
        acc[mt][0][3] = fmaf(tmp[mt][0][3], f1, acc[mt][0][3]);
      }
      __syncwarp();
    }
    if (stuck) {  // what else was asked for lands before the warp goes on
      if (lane == 0) {
        raise_flag(a.c.status, ENTMAXKV_DEV_TIMEOUT);
        for (int n = used; n < used + mine; ++n) mbar_wait_bounded(&bars[warp][n & 1], (uint32_t)(n >> 1) & 1u);
      }
      __syncwarp();
    }
    if (__syncthreads_or(stuck)) break;  // (and the list is done with)
    used += mine;
  }
  __syncthreads();
  // the warps' sums, in order, through the slabs' place (they are done with)
  float* red = reinterpret_cast<float*>(base_p);  // [NW][8][D]
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (2 * c + j < G)
        *reinterpret_cast<float2*>(red + (warp * 8 + 2 * c + j) * D + 16 * mt + 2 * r) =
            make_float2(acc[mt][0][j], acc[mt][0][2 + j]);
  __syncthreads();
  for (int i = tid; i < G * D; i += NTH) {
    float v = 0.0f;
#pragma unroll
    for (int wp = 0; wp < NW; ++wp) v += red[wp * 8 * D + i];
    part[i] = v;
  }
  cluster_sync();
  // each block adds up its share of the outputs
  const int per = (G * D + C - 1) / C;
  for (int i = rank * per + tid; i < min(G * D, (rank + 1) * per); i += NTH) {
    float v = 0.0f;
    for (int k = 0; k < C; ++k) v += peer_load(peer(smem_u32(&part[i]), k));
    if (isnan(tau_sh[i / D].b)) v = CUDART_NAN_F;
    a.out.p[(long long)s.start * a.out.ts + (long long)(kvh * G + i / D) * a.out.hs + i % D] = __float2bfloat16_rn(v);
  }
  cluster_sync();  // no block leaves while its sums are read
}

static size_t up256e(size_t x) { return (x + 255) & ~(size_t)255; }
// Tiles of the line: a slot's pages, rounded up to whole tiles.
static size_t ent_line(const entmaxkv_config& cfg, int n_seqs) {
  const size_t pages = cfg.max_pages_per_seq, per = kEntKeys / cfg.page_size;
  return (size_t)n_seqs * cfg.num_kv_heads * ((pages + per - 1) / per);
}

size_t attend_entmax_bytes(const entmaxkv_config& cfg, int n_seqs) {
  const size_t line = ent_line(cfg, n_seqs);
  return up256e((size_t)n_seqs * sizeof(EntUnit)) + up256e(line * cfg.group * kEntKeys * 4) + up256e(line * cfg.group * 4);
}

template <bool I8, int D, int P>
static cudaError_t entmax_t(EntArgs& e, int sms, cudaStream_t st) {
  const Q8AttendArgs& a = e.a;
  const int smem1 = kScoreWarps * kScoreSlabs * kEntKeys * D + 1024;
  // the scores handed round, V slabs with the list behind them, and the warps' sums take turns
  const int sent = kEntCluster * kEntWarps * kEntSent * 4, slabs = 2 * kEntWarps * kEntKeys * D + kEntList * 4;
  const int red = kEntWarps * 8 * D * 4, smem2 = max(sent, max(slabs, red)) + 1024;
  cudaError_t err = ensure_smem((const void*)ent_score_kernel<I8, D, P>, smem1);
  if (err == cudaSuccess) err = ensure_smem((const void*)ent_finish_kernel<I8, D, P>, smem2);
  if (err != cudaSuccess) return err;
  CUtensorMap km, vm;
  if ((err = make_q8_map(&km, a.c.k_pool, a.c.nphys, a.c.Hkv, P, D)) != cudaSuccess) return err;
  if ((err = make_q8_map(&vm, a.c.v_pool, a.c.nphys, a.c.Hkv, P, D)) != cudaSuccess) return err;
  err = launch_k(true, ent_score_kernel<I8, D, P>, dim3(sms), dim3(kScoreWarps * 32), (size_t)smem1, st, e, km);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  // as many blocks a unit as there are multiprocessors for, in one wave
  int cl = kEntCluster;
  while (cl > 1 && (long long)cl * a.c.Hkv * a.b.n_seqs > sms) cl >>= 1;
  cfg.gridDim = dim3(cl, a.c.Hkv, a.b.n_seqs);
  cfg.blockDim = dim3(kEntWarps * 32);
  cfg.dynamicSmemBytes = (size_t)smem2;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ent_finish_kernel<I8, D, P>, e, vm);
}

template <bool I8>
static cudaError_t entmax_d(EntArgs& e, int sms, cudaStream_t st) {
  if (e.a.c.D == 128) return e.a.c.P == 32 ? entmax_t<I8, 128, 32>(e, sms, st) : entmax_t<I8, 128, 16>(e, sms, st);
  return e.a.c.P == 32 ? entmax_t<I8, 64, 32>(e, sms, st) : entmax_t<I8, 64, 16>(e, sms, st);
}

cudaError_t launch_attend_entmax(const entmaxkv_config& cfg, Q8AttendArgs a, bool i8, float alpha, void* ws, int sms,
                                 cudaStream_t st) {
  EntArgs e;
  e.a1 = alpha - 1.0f;
  e.beta = (float)(1.0 / ((double)alpha - 1.0));
  const size_t line = ent_line(cfg, a.b.n_seqs);
  char* p = static_cast<char*>(ws);
  e.slots = reinterpret_cast<EntUnit*>(p);
  p += up256e((size_t)a.b.n_seqs * sizeof(EntUnit));
  e.z = reinterpret_cast<float*>(p);
  p += up256e(line * a.c.G * kEntKeys * 4);
  e.pmax = reinterpret_cast<float*>(p);
  e.a = a;
  return i8 ? entmax_d<true>(e, sms, st) : entmax_d<false>(e, sms, st);
}

}  // namespace ekv
