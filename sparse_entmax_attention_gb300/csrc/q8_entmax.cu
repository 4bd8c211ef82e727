// q8_entmax.cu -- alpha-entmax decode over the 8-bit paged cache, one new token
// a sequence.
//
//   z_j = (α−1)·s_j,  Σ_j [z_j − τ]_+^β = 1 (β = 1/(α−1)),  o = Σ_j [z_j − τ]_+^β v_j.
//
// 1. score: K streams once, on the same line of pages as the softmax kernel;
//    z and each page's largest z go to the workspace.
// 2. solve: a block per (slot, query head). No token at or below z_max − 1 can
//    carry weight (τ ≥ z_max − 1, where the sum is at least 1), so only pages
//    whose largest z clears that are looked at again. Newton steps from there
//    stay below the root of the convex, falling sum, and after each the
//    closed-form root on the support so far is taken once it lies within it.
// 3. weigh: V is read for pages with some z above its head's τ only; p is
//    rounded to halves against its page's largest p. 4. join the splits.
#include "q8_tiles.cuh"

namespace ekv {

constexpr int kEntWarps = 8;
constexpr int kEntStages = 4;
constexpr int kEntSplits = 64;
constexpr int kSolveThreads = 512;
constexpr int kSolvePages = 8192;  // candidate pages a solving block lists

struct EntArgs {
  Q8AttendArgs a;
  float alpha, a1, beta;
  float* z;       // [line page][G][P]
  float* pmax;    // [line page][G]
  float2* tau;    // [slot][Hq] τ as a sum of two floats
  float* part;    // [unit][splits][G][D]
  int splits;
};

__device__ __forceinline__ Q8Span ent_span(const Q8AttendArgs& a, const Q8Slot& s, int b) {
  return q8_span(a.c, a.sc, s, b, 0, 1);
}

template <bool I8, int D, int P>
__global__ void __launch_bounds__(kEntWarps * 32, 1)
    ent_score_kernel(EntArgs e, const __grid_constant__ CUtensorMap kmap) {
  pdl_enter();
  constexpr int NW = kEntWarps, ST = kEntStages, SLAB = P * D;
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
        return s.count > 0 ? (long long)ent_span(a, s, b).T * Hkv : 0LL;
      },
      [&](int b, long long where) { a.cum[b] = where; });
  const long long w_begin = at.begin, w_end = at.end;
  if (w_begin >= w_end) return;
  const int r = lane >> 2, c = lane & 3;
  int slot = at.slot;
  long long cum = at.cum, w = w_begin;
  int filled = 0, used = 0;
  bool stuck = false;
  while (w < w_end && !stuck) {
    const Q8Slot s = q8_slot(a.c, a.b, slot, nullptr);
    const Q8Span sp = s.count > 0 ? ent_span(a, s, slot) : Q8Span{0, 0, 0, 0, 0};
    const int T = sp.T;
    if (w >= cum + (long long)T * Hkv) {
      cum += (long long)T * Hkv;
      ++slot;
      continue;
    }
    const long long off = w - cum;
    const int kvh = (int)div_line(off, T), t0 = (int)(off - (long long)kvh * T);
    const int n = (int)min((long long)(T - t0), w_end - w);
    uint32_t bq[1][D / 16][2];
    Q8Row row[2];
    float inv;
    uint4 qw[D / 32];
    q_load<D>(r < G ? a.q.p + (long long)s.start * a.q.ts + (long long)(kvh * G + r) * a.q.hs : nullptr, lane, qw);
    q_half_frag<D>(qw, bq[0], inv);
    const int pos = s.L - 1;
    int lo = a.sc.window > 0 ? max(0, pos - a.sc.window + 1) : 0;
    if (a.sc.first_key) lo = max(lo, a.sc.first_key[s.start]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      row[j].cs = q8_row_scale(__shfl_sync(0xffffffffu, inv, (2 * c + j) * 4), a.sc, e.a1);
      row[j].slope = a.sc.slopes && 2 * c + j < G ? a.sc.slopes[kvh * G + 2 * c + j] * e.a1 : 0.0f;
      row[j].pos = pos;
      row[j].lo = lo;
    }
    for (int p0 = 0; p0 < n && !stuck; p0 += 32) {
      const int pn = min(32, n - p0);
      int ph = -1;
      float ks_l = 0.0f;
      if (lane < pn) {
        ph = phys_page(a.c.block_table, s.seq, sp.page(t0 + p0 + lane), a.c.maxp, a.c.nphys, a.c.status);
        if (ph >= 0) ks_l = a.c.k_scale[(size_t)ph * Hkv + kvh];
      }
      int ask = 0;
      auto refill = [&]() {
        while (ask < pn && filled - used < ST) {
          const int f = __shfl_sync(0xffffffffu, ph, ask);
          ++ask;
          if (f < 0) continue;
          const int sg = filled % ST;
          if (lane == 0) {
            mbar_expect_tx(&bars[warp][sg], SLAB);
            tma_load_3d(ring_p + sg * SLAB, &kmap, 0, kvh * P, f, &bars[warp][sg]);
          }
          ++filled;
        }
      };
      refill();
      for (int i = 0; i < pn; ++i) {
        const size_t line = (size_t)(w + p0 + i);
        float* zo = e.z + line * G * P;
        const bool there = __shfl_sync(0xffffffffu, ph, i) >= 0;
        const float ks = __shfl_sync(0xffffffffu, ks_l, i);
        const int sg = used % ST;
        if (there && !__all_sync(0xffffffffu, mbar_wait_bounded(&bars[warp][sg], (used / ST) & 1))) {
          stuck = true;
          break;
        }
        const int key0 = sp.page(t0 + p0 + i) * P;
        const bool whole = (key0 + P - 1 <= pos && key0 >= lo) || key0 + P <= sp.pre;
        float pm[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int mt = 0; mt < P / 16; ++mt) {
          float acc[1][4] = {{0.f, 0.f, 0.f, 0.f}};
          if (there) k_dot<I8, D, 1>(ring + sg * SLAB, 16 * mt, lane, bq, acc);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int tk = 16 * mt + r, h = 2 * c + j;
            const float dot[2] = {acc[0][j], acc[0][2 + j]};
            float v[2];
            q8_scores(dot, v, row[j], ks, key0 + tk, a.sc, e.a1, 0.0f);
            if (!there || (!whole && !q8_sees(row[j], key0 + tk, sp.pre))) v[0] = -CUDART_INF_F;
            if (!there || (!whole && !q8_sees(row[j], key0 + tk + 8, sp.pre))) v[1] = -CUDART_INF_F;
            if (h < G) {
              zo[h * P + tk] = v[0];
              zo[h * P + tk + 8] = v[1];
            }
            pm[j] = max3(pm[j], v[0], v[1]);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          pm[j] = fmaxf(pm[j], __shfl_xor_sync(0xffffffffu, pm[j], 4));
          pm[j] = fmaxf(pm[j], __shfl_xor_sync(0xffffffffu, pm[j], 8));
          pm[j] = fmaxf(pm[j], __shfl_xor_sync(0xffffffffu, pm[j], 16));
          if (r == 0 && 2 * c + j < G) e.pmax[line * G + 2 * c + j] = pm[j];
        }
        if (there) {
          __syncwarp();
          ++used;
          refill();
        }
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

// Block sums of four values and a minimum.
__device__ __forceinline__ void block_sums(float (&v)[4], float& mn, float (*sh)[5]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = warp_sum(v[i]);
  mn = warp_min_f(mn);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sh[warp][i] = v[i];
    sh[warp][4] = mn;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float t = 0.0f;
    for (int w = 0; w < kSolveThreads / 32; ++w) t += sh[w][i];
    v[i] = t;
  }
  mn = CUDART_INF_F;
  for (int w = 0; w < kSolveThreads / 32; ++w) mn = fminf(mn, sh[w][4]);
  __syncthreads();
}

template <int P>
__global__ void __launch_bounds__(kSolveThreads) ent_solve_kernel(EntArgs e) {
  pdl_enter();
  __shared__ int list[kSolvePages];
  __shared__ float sh[kSolveThreads / 32][5];
  __shared__ int sh_scan[32];
  const Q8AttendArgs& a = e.a;
  const int b = blockIdx.y, h = blockIdx.x, G = a.c.G, kvh = h / G, g = h - kvh * G, tid = threadIdx.x;
  const Q8Slot s = q8_slot(a.c, a.b, b, nullptr);
  if (s.count == 0) return;
  const int Hq = a.c.Hkv * G;
  const int T = ent_span(a, s, b).T;
  const size_t line0 = (size_t)(a.cum[b] + (long long)kvh * T);
  const float* pmax = e.pmax + line0 * G + g;
  float top = -CUDART_INF_F;
  for (int t = tid; t < T; t += kSolveThreads) top = fmaxf(top, pmax[(size_t)t * G]);
  {
    float v[4] = {0.f, 0.f, 0.f, 0.f}, mn = -top;
    block_sums(v, mn, sh);
    top = -mn;
  }
  float* tau_out = a.tau ? a.tau + (size_t)s.start * Hq + h : nullptr;
  float2* tau_ws = e.tau + (size_t)b * Hq + h;
  if (!(top > -CUDART_INF_F)) {
    if (tid == 0) {
      *tau_ws = make_float2(CUDART_NAN_F, 0.0f);
      if (tau_out) *tau_out = CUDART_NAN_F;
    }
    return;
  }
  const float T0 = top - 1.0f;
  // pages that can carry weight, in order
  int np = 0;
  for (int t0 = 0; t0 < T; t0 += kSolveThreads) {
    const int t = t0 + tid;
    const bool in = t < T && pmax[(size_t)t * G] > T0;
    int total;
    const int at = np + block_exclusive_scan(in ? 1 : 0, sh_scan, total);
    if (in && at < kSolvePages) list[at] = t;
    np += total;
  }
  const bool big = np > kSolvePages;  // walk every page instead
  const int walk = big ? T : np;
  __syncthreads();
  const float* zb = e.z + (line0 * G + g) * P;  // page t's scores at zb + t·G·P
  const bool b2 = e.beta == 2.0f, b1 = e.beta == 1.0f;
  double tau = (double)T0, lo = (double)T0, hi = (double)top;
  bool done = false;
  for (int it = 0; it < 100 && !done; ++it) {
    const float th = (float)tau, tl = (float)(tau - (double)th);
    float v[4] = {0.f, 0.f, 0.f, 0.f}, mn = CUDART_INF_F;
    for (int i = tid; i < walk * P; i += kSolveThreads) {
      const int t = big ? i / P : list[i / P];
      const float y = (zb[(size_t)t * G * P + i % P] - th) - tl;
      if (y > 0.0f) {
        v[0] += 1.0f;
        mn = fminf(mn, y);
        if (b2 || b1) {
          v[1] += y;
          v[2] = fmaf(y, y, v[2]);
        } else {
          v[1] += powf(y, e.beta - 1.0f);
          v[2] += powf(y, e.beta);
        }
      }
    }
    block_sums(v, mn, sh);
    const float k = v[0];
    const float tol = 1e-7f * fmaxf(1.0f, fabsf((float)tau));
    if (b2 || b1) {
      const float s1 = v[1], s2 = v[2];
      float d, step;
      if (b2) {  // Σ(y − δ)² = 1 with δ ≤ min y, written without cancellation
        const float disc = s1 * s1 - k * (s2 - 1.0f);
        d = disc >= 0.0f ? (s2 - 1.0f) / (s1 + sqrtf(disc)) : CUDART_INF_F;
        step = (s2 - 1.0f) / (2.0f * s1);
      } else {
        d = step = (s1 - 1.0f) / k;
      }
      if (!(k > 0.0f)) break;
      if (d >= -1e-7f && d <= mn * (1.0f + 1e-6f) + 1e-7f) {
        tau += (double)d;
        done = true;
      } else if (!(step > tol)) {
        if (step > 0.0f) tau += (double)step;
        done = true;
      } else {
        tau += (double)step;
      }
    } else {  // any order: Newton inside a bracket kept by the sign of the sum − 1
      const float sb1 = v[1], sb = v[2];
      if (k == 0.0f || sb < 1.0f) hi = tau;
      else lo = tau;
      double nt = 0.5 * (lo + hi);
      if (k > 0.0f) {
        const float step = (sb - 1.0f) / (e.beta * sb1);
        if (fabsf(step) <= tol) {
          tau += (double)step;
          done = true;
          continue;
        }
        if (tau + (double)step > lo && tau + (double)step < hi) nt = tau + (double)step;
      }
      tau = nt;
      if (hi - lo <= (double)tol) done = true;
    }
  }
  if (tid == 0) {
    if (!done) raise_flag(a.c.status, ENTMAXKV_DEV_TAU_NOCONV);
    const float th = (float)tau;
    *tau_ws = make_float2(th, (float)(tau - (double)th));
    if (tau_out) *tau_out = th;
  }
}

// Block (split, unit, slot): its share of the unit's pages, a warp a page.
template <bool I8, int D, int P>
__global__ void __launch_bounds__(kEntWarps * 32)
    ent_weigh_kernel(EntArgs e, const __grid_constant__ CUtensorMap vmap) {
  pdl_enter();
  constexpr int NW = kEntWarps, SLAB = P * D;
  extern __shared__ __align__(128) unsigned char dyn_sm[];
  __shared__ uint64_t bars[NW];
  const Q8AttendArgs& a = e.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z, G = a.c.G, Hkv = a.c.Hkv;
  const Q8Slot s = q8_slot(a.c, a.b, b, nullptr);
  if (s.count == 0) return;
  const uint32_t base = (smem_u32(dyn_sm) + 1023u) & ~1023u;
  const uint32_t slab = base + warp * SLAB;
  unsigned char* slab_p = dyn_sm + (slab - smem_u32(dyn_sm));
  if (lane == 0) {
    mbar_init(&bars[warp], 1);
    mbar_fence_init();
  }
  __syncwarp();
  const Q8Span sp = ent_span(a, s, b);
  const int T = sp.T;
  const size_t line0 = (size_t)(a.cum[b] + (long long)kvh * T);
  const int lo = (int)((long long)T * split / e.splits), hi = (int)((long long)T * (split + 1) / e.splits);
  const int r = lane >> 2, c = lane & 3;
  const float2 tau = r < G ? e.tau[(size_t)b * Hkv * G + kvh * G + r] : make_float2(CUDART_INF_F, 0.0f);
  const float nan_off = tau.x;
  float acc[D / 16][1][4];
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) acc[mt][0][0] = acc[mt][0][1] = acc[mt][0][2] = acc[mt][0][3] = 0.0f;
  uint32_t phase = 0u;
  bool stuck = false;
  for (int t = lo + warp; t < hi && !stuck; t += NW) {
    // the largest y = z − τ of this page for row r
    float ym = -1.0f;
    if (r < G) ym = (e.pmax[(line0 + t) * G + r] - nan_off) - tau.y;
    if (!__any_sync(0xffffffffu, ym > 0.0f)) continue;
    const int page = sp.page(t);
    const int ph = phys_page(a.c.block_table, s.seq, page, a.c.maxp, a.c.nphys, nullptr);
    if (ph < 0) continue;
    if (lane == 0) {
      mbar_expect_tx(&bars[warp], SLAB);
      tma_load_3d(slab_p, &vmap, 0, kvh * P, ph, &bars[warp]);
    }
    const float vs = a.c.v_scale[(size_t)ph * Hkv + kvh];
    // the page's weights against a power of two above its largest
    const float big = ym > 0.0f ? pos_pow(ym, e.beta) : 0.0f;
    const int ex = min(max((int)(__float_as_uint(big) >> 23) - 126, -100), 100);
    const float up = __uint_as_float((uint32_t)(127 - ex) << 23), down = __uint_as_float((uint32_t)(127 + ex) << 23);
    uint32_t bf[P / 16][1][2];
#pragma unroll
    for (int kt = 0; kt < P / 16; ++kt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float2 z = make_float2(-CUDART_INF_F, -CUDART_INF_F);
        if (ym > 0.0f)
          z = *reinterpret_cast<const float2*>(e.z + ((line0 + t) * G + r) * P + 16 * kt + 8 * j + 2 * c);
        const float y0 = (z.x - tau.x) - tau.y, y1 = (z.y - tau.x) - tau.y;
        const __half2 p = __floats2half2_rn(y0 > 0.0f ? pos_pow(y0, e.beta) * up : 0.0f,
                                            y1 > 0.0f ? pos_pow(y1, e.beta) * up : 0.0f);
        bf[kt][0][j] = *reinterpret_cast<const uint32_t*>(&p);
      }
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bars[warp], phase))) {
      stuck = true;
      break;
    }
    phase ^= 1u;
    const int nv = s.L - page * P;
    if (nv < P) {
      for (int i = lane; i < (P - nv) * (D / 16); i += 32)
        *reinterpret_cast<uint4*>(slab_p + nv * D + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      __syncwarp();
    }
    float tmp[D / 16][1][4];
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) tmp[mt][0][0] = tmp[mt][0][1] = tmp[mt][0][2] = tmp[mt][0][3] = 0.0f;
#pragma unroll
    for (int kt = 0; kt < P / 16; ++kt) v_dot<I8, D, 1>(slab, 16 * kt, lane, bf[kt], tmp);
    const float f0 = __shfl_sync(0xffffffffu, down, 8 * c) * vs, f1 = __shfl_sync(0xffffffffu, down, 8 * c + 4) * vs;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      acc[mt][0][0] = fmaf(tmp[mt][0][0], f0, acc[mt][0][0]);
      acc[mt][0][2] = fmaf(tmp[mt][0][2], f0, acc[mt][0][2]);
      acc[mt][0][1] = fmaf(tmp[mt][0][1], f1, acc[mt][0][1]);
      acc[mt][0][3] = fmaf(tmp[mt][0][3], f1, acc[mt][0][3]);
    }
    __syncwarp();
  }
  if (stuck && lane == 0) {
    raise_flag(a.c.status, ENTMAXKV_DEV_TIMEOUT);
    mbar_wait_bounded(&bars[warp], phase);
  }
  __syncthreads();
  // the warps' sums, in order, through shared memory (the slabs are done with)
  float* red = reinterpret_cast<float*>(dyn_sm + (base - smem_u32(dyn_sm)));  // [NW][8][D]
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<float2*>(red + (warp * 8 + 2 * c + j) * D + 16 * mt + 2 * r) =
          make_float2(acc[mt][0][j], acc[mt][0][2 + j]);
  __syncthreads();
  for (int i = tid; i < G * D; i += NW * 32) {
    float v = 0.0f;
    for (int wp = 0; wp < NW; ++wp) v += red[wp * 8 * D + i];
    if (e.splits == 1)
      a.out.p[(long long)s.start * a.out.ts + (long long)(kvh * G + i / D) * a.out.hs + i % D] = __float2bfloat16_rn(v);
    else
      e.part[(((size_t)b * Hkv + kvh) * e.splits + split) * G * D + i] = v;
  }
}

__global__ void __launch_bounds__(256) ent_join_kernel(EntArgs e) {
  pdl_enter();
  const Q8AttendArgs& a = e.a;
  const int kvh = blockIdx.x, b = blockIdx.y, G = a.c.G, D = a.c.D;
  const Q8Slot s = q8_slot(a.c, a.b, b, nullptr);
  if (s.count == 0) return;
  for (int i = threadIdx.x; i < G * D; i += 256) {
    float v = 0.0f;
    for (int sp = 0; sp < e.splits; ++sp) v += e.part[(((size_t)b * a.c.Hkv + kvh) * e.splits + sp) * G * D + i];
    a.out.p[(long long)s.start * a.out.ts + (long long)(kvh * G + i / D) * a.out.hs + i % D] = __float2bfloat16_rn(v);
  }
}

static size_t up256e(size_t x) { return (x + 255) & ~(size_t)255; }

size_t attend_entmax_bytes(const entmaxkv_config& cfg, int n_seqs) {
  const size_t line = (size_t)n_seqs * cfg.num_kv_heads * cfg.max_pages_per_seq;
  const size_t Hq = (size_t)cfg.num_kv_heads * cfg.group;
  return up256e((size_t)(n_seqs + 1) * 8) + up256e(line * cfg.group * cfg.page_size * 4) + up256e(line * cfg.group * 4) +
         up256e((size_t)n_seqs * Hq * 8) + up256e((size_t)n_seqs * Hq * kEntSplits * cfg.head_dim * 4);
}

template <bool I8, int D, int P>
static cudaError_t entmax_t(EntArgs& e, int sms, cudaStream_t st) {
  const Q8AttendArgs& a = e.a;
  const int smem1 = kEntWarps * kEntStages * P * D + 1024;
  const int red = kEntWarps * 8 * D * 4, slabs = kEntWarps * P * D;
  const int smem3 = (red > slabs ? red : slabs) + 1024;
  cudaError_t err = ensure_smem((const void*)ent_score_kernel<I8, D, P>, smem1);
  if (err == cudaSuccess) err = ensure_smem((const void*)ent_weigh_kernel<I8, D, P>, smem3);
  if (err != cudaSuccess) return err;
  CUtensorMap km, vm;
  if ((err = make_q8_map(&km, a.c.k_pool, a.c.nphys, a.c.Hkv, P, D)) != cudaSuccess) return err;
  if ((err = make_q8_map(&vm, a.c.v_pool, a.c.nphys, a.c.Hkv, P, D)) != cudaSuccess) return err;
  err = launch_k(false, ent_score_kernel<I8, D, P>, dim3(sms), dim3(kEntWarps * 32), (size_t)smem1, st, e, km);
  if (err != cudaSuccess) return err;
  err = launch_k(false, ent_solve_kernel<P>, dim3(a.c.Hkv * a.c.G, a.b.n_seqs), dim3(kSolveThreads), 0, st, e);
  if (err != cudaSuccess) return err;
  err = launch_k(false, ent_weigh_kernel<I8, D, P>, dim3(e.splits, a.c.Hkv, a.b.n_seqs), dim3(kEntWarps * 32),
                 (size_t)smem3, st, e, vm);
  if (err != cudaSuccess || e.splits == 1) return err;
  return launch_k(false, ent_join_kernel, dim3(a.c.Hkv, a.b.n_seqs), dim3(256), 0, st, e);
}

template <bool I8>
static cudaError_t entmax_d(EntArgs& e, int sms, cudaStream_t st) {
  if (e.a.c.D == 128) return e.a.c.P == 32 ? entmax_t<I8, 128, 32>(e, sms, st) : entmax_t<I8, 128, 16>(e, sms, st);
  return e.a.c.P == 32 ? entmax_t<I8, 64, 32>(e, sms, st) : entmax_t<I8, 64, 16>(e, sms, st);
}

cudaError_t launch_attend_entmax(Q8AttendArgs a, bool i8, float alpha, void* ws, int sms, cudaStream_t st) {
  EntArgs e;
  e.alpha = alpha;
  e.a1 = alpha - 1.0f;
  e.beta = (float)(1.0 / ((double)alpha - 1.0));
  const int S = a.b.n_seqs, G = a.c.G;
  const size_t line = (size_t)S * a.c.Hkv * a.c.maxp, Hq = (size_t)a.c.Hkv * G;
  char* p = static_cast<char*>(ws);
  a.cum = reinterpret_cast<long long*>(p);
  p += up256e((size_t)(S + 1) * 8);
  e.z = reinterpret_cast<float*>(p);
  p += up256e(line * G * a.c.P * 4);
  e.pmax = reinterpret_cast<float*>(p);
  p += up256e(line * G * 4);
  e.tau = reinterpret_cast<float2*>(p);
  p += up256e((size_t)S * Hq * 8);
  e.part = reinterpret_cast<float*>(p);
  const long long units = (long long)S * a.c.Hkv;
  e.splits = (int)max(1LL, min((long long)kEntSplits, (4LL * sms + units - 1) / units));
  e.a = a;
  return i8 ? entmax_d<true>(e, sms, st) : entmax_d<false>(e, sms, st);
}

}  // namespace ekv
