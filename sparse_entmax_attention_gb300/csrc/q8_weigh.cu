// q8_weigh.cu -- the weight that a few rows a sequence give to the keys of the
// 8-bit paged cache.
//
//   w_j ← decay·w_j + Σ over rows and heads of coef·p_j,
//   p_j = e^{s_j − tau}  or  [(α−1)·s_j − tau]_+^{1/(α−1)},
//
// scores, masks and statistics (tau) as attention forms them. Keys from L − fresh
// on begin at 0. Everything is there before a key is met, so a tile of keys is
// answered by whoever holds it: no pass is joined with another, and every sum has
// one order.
//
// Up to 32 rows a sequence (max_count · group). Bound: K's bytes. As in the streaming attention, the tiles (32 keys) of all
// (slot, KV head) units form one line cut into equal pieces for all warps of the
// device, and a warp streams its K pages through a ring of tensor copies:
//   S = K·q^T   m16n8k16 in halves, 16 keys × 8 rows a product, fp32 sums;
//   p           in fp32, summed over a lane's rows and the four lanes of a key.
//
// Measured: 16 sequences of 1000-32000 tokens, 8 KV heads of 4 query heads, d = 128, e4m3, entmax (165 MB): 38 us,
// 4.3 TB/s, 0.64 of the measured copy (45 with a key's weight asked for in its own tile); 16 of 24000, int8 (418 MB):
// 75 us, 5.5 TB/s, codes to halves beside it (ALU 55%, IPC 2.4). One sequence of 32768 (36 MB): 13-15 us, of which the
// bytes are 5.3: start, and three or four tiles a warp.
#include "q8_tiles.cuh"

namespace ekv {

constexpr int kWeighKeys = 32;
// Warps of a block: four tiles of 8 rows need twice the registers.
template <int NT>
constexpr int kWeighWarps = NT == 4 ? 8 : 16;
template <int D, int NT>
constexpr int kWeighSlabs = 192 * 1024 / (kWeighWarps<NT> * kWeighKeys * D);

// A slot's pages: those of the span, and what changes beside it (faded or fresh
// weights). T tiles on the line a KV head.
struct WeighSlot {
  Q8Slot s;
  Q8Span sp;    // keys that are seen
  int npre, wfirst, fresh;  // pages on the line: [0, npre) and [wfirst, sp.npages); first fresh key
  int T;
  __device__ __forceinline__ int page(int t) const { return t < npre ? t : t - npre + wfirst; }
  __device__ __forceinline__ int pages() const { return npre + sp.npages - wfirst; }
  __device__ __forceinline__ bool seen(int page) const { return page < sp.npre || page >= sp.wfirst; }
};
__device__ __forceinline__ WeighSlot weigh_slot(const Q8WeighArgs& a, int b, uint32_t* st) {
  WeighSlot x;
  x.s = q8_slot(a.c, a.b, b, st);
  x.sp = Q8Span{0, 0, 0, 0, 0};
  x.npre = x.wfirst = x.fresh = x.T = 0;
  if (x.s.count > 0) {
    x.sp = q8_span(a.c, a.sc, x.s, b, 0, x.s.count);
    x.fresh = x.s.L - min(max(a.fresh ? a.fresh[b] : x.s.count, 0), x.s.L);
    x.wfirst = a.decay != 1.0f ? 0 : min(x.sp.wfirst, x.fresh / a.c.P);
    x.npre = min(x.sp.npre, x.wfirst);
    x.T = (x.pages() * a.c.P + kWeighKeys - 1) / kWeighKeys;
  }
  return x;
}

template <bool I8, int D, int P, int NT, bool ENT>
__global__ void __launch_bounds__(kWeighWarps<NT> * 32, 1) weigh_kernel(Q8WeighArgs a, const __grid_constant__ CUtensorMap kmap) {
  pdl_enter();
  constexpr int NW = kWeighWarps<NT>, ST = kWeighSlabs<D, NT>, SLAB = kWeighKeys * D, PP = kWeighKeys / P;
  extern __shared__ __align__(128) unsigned char dyn_sm[];
  __shared__ uint64_t bars[NW][ST];
  __shared__ LineSmem<NW> sh_line;
  constexpr int kFew = 256;
  __shared__ WeighSlot sh_info[kFew];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = ((smem_u32(dyn_sm) + 1023u) & ~1023u) + (uint32_t)warp * ST * SLAB;
  unsigned char* ring_p = dyn_sm + (ring - smem_u32(dyn_sm));
  if (lane == 0) {
    for (int i = 0; i < ST; ++i) mbar_init(&bars[warp][i], 1);
    mbar_fence_init();
  }
  if (tid == 0) prefetch_map(&kmap);
  const int n_seqs = a.b.n_seqs;
  const bool few = n_seqs <= kFew;
  const LinePlace at = line_place<NW>(
      n_seqs, a.c.status, sh_line,
      [&](int b, uint32_t* st) {
        const WeighSlot x = weigh_slot(a, b, st);
        if (few) sh_info[b] = x;
        return (long long)x.T * a.c.Hkv;
      },
      [](int, long long) {});
  const int G = a.c.G, Hkv = a.c.Hkv;
  const int r = lane >> 2, c = lane & 3;
  const float unit = ENT ? a.a1 : kLog2e;
  int slot = at.slot;
  long long cum = at.cum, w = at.begin;
  int filled = 0, used = 0;
  bool stuck = false;
  while (w < at.end && !stuck) {
    const WeighSlot x = few ? sh_info[slot] : weigh_slot(a, slot, nullptr);
    if (w >= cum + (long long)x.T * Hkv) {
      cum += (long long)x.T * Hkv;
      ++slot;
      continue;
    }
    const long long off = w - cum;
    const int kvh = (int)div_line(off, x.T), t0 = (int)(off - (long long)kvh * x.T);
    const int n = (int)min((long long)(x.T - t0), at.end - w);
    const int n_rows = x.s.count * G, n_pages = x.pages();
    // 32 tiles' places and scales at once, a tile a lane
    int ph[PP];
    float ks_l[PP];
    auto look_up = [&](int p0) {
#pragma unroll
      for (int q = 0; q < PP; ++q) {
        const int t = (t0 + p0 + lane) * PP + q;
        ph[q] = -1;
        ks_l[q] = 0.0f;
        if (p0 + lane < n && t < n_pages) {
          ph[q] = phys_page(a.c.block_table, x.s.seq, x.page(t), a.c.maxp, a.c.nphys, a.c.status);
          if (ph[q] >= 0) ks_l[q] = a.c.k_scale[(size_t)ph[q] * Hkv + kvh];
        }
      }
    };
    int ask = 0;
    auto refill = [&](int end) {
      while (ask < end && filled - used < ST) {
        int f[PP], there = 0;
#pragma unroll
        for (int q = 0; q < PP; ++q) {
          f[q] = __shfl_sync(0xffffffffu, ph[q], ask & 31);
          if (!x.seen(x.page((t0 + ask) * PP + q))) f[q] = -1;
          there += f[q] >= 0;
        }
        ++ask;
        if (!there) continue;
        const int sg = filled % ST;
        if (lane == 0) {
          mbar_expect_tx(&bars[warp][sg], (uint32_t)(there * P * D));
#pragma unroll
          for (int q = 0; q < PP; ++q)
            if (f[q] >= 0) tma_load_3d(ring_p + sg * SLAB + q * P * D, &kmap, 0, kvh * P, f[q], &bars[warp][sg]);
        }
        ++filled;
      }
    };
    // the slot's rows: queries, and what turns a score into a weight
    uint32_t bq[NT][D / 16][2];
    Q8Row row[NT][2];
    float add[NT][2], cf[NT][2];
    int pos_min = 0x7fffffff, lo_max = 0;
    {
      uint4 qw[NT][D / 32];
      float t[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t rj = 8 * nt + 2 * c + j, i = rj / (uint32_t)G;
          const int h = kvh * G + (int)(rj - i * G);
          Q8Row& q = row[nt][j];
          q.slope = 0.0f;
          q.pos = -1;
          q.lo = 0;
          t[nt][j] = CUDART_NAN_F;
          cf[nt][j] = 0.0f;
          if ((int)rj < n_rows) {
            const long long tok = x.s.start + (int)i;
            t[nt][j] = a.tau[tok * Hkv * G + h];
            cf[nt][j] = a.coef ? a.coef[tok * Hkv * G + h] : 1.0f;
            q.pos = x.s.L - x.s.count + (int)i;
            if (a.sc.window > 0) q.lo = max(0, q.pos - a.sc.window + 1);
            if (a.sc.first_key) q.lo = max(q.lo, a.sc.first_key[tok]);
            if (a.sc.slopes) q.slope = a.sc.slopes[h] * unit;
            pos_min = min(pos_min, q.pos);
            lo_max = max(lo_max, q.lo);
          }
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t rho = 8 * nt + r, tok = rho / (uint32_t)G;
        q_load<D>((int)rho < n_rows ? a.q.p + (long long)(x.s.start + (int)tok) * a.q.ts +
                                          (long long)(kvh * G + (int)(rho - tok * G)) * a.q.hs
                                    : nullptr,
                  lane, qw[nt]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float inv;
        q_half_frag<D>(qw[nt], bq[nt], inv);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          row[nt][j].cs = q8_row_scale(__shfl_sync(0xffffffffu, inv, (2 * c + j) * 4), a.sc, unit);
          // a row without a statistic, or that does not count, adds nothing
          const bool counts = fabsf(t[nt][j]) < CUDART_INF_F && cf[nt][j] > 0.0f;
          if (!counts) cf[nt][j] = 0.0f;
          add[nt][j] = counts ? -t[nt][j] * (ENT ? 1.0f : kLog2e) : 0.0f;
        }
      }
      pos_min = __reduce_min_sync(0xffffffffu, pos_min);
      lo_max = __reduce_max_sync(0xffffffffu, lo_max);
    }
    look_up(0);
    refill(min(n, 32));
    // the lane's key of tile i (key 8c + r), and what it gathered; asked for a tile ahead, as the load takes longer than
    // a tile's products
    struct Place {
      float* p;
      float before;
      bool there;
    };
    auto place = [&](int i) -> Place {
      const bool second = PP == 2 && c >= 2;
      int f = __shfl_sync(0xffffffffu, ph[0], i & 31);
      if (PP == 2) {
        const int g = __shfl_sync(0xffffffffu, ph[PP - 1], i & 31);
        if (second) f = g;
      }
      const int key = x.page((t0 + i) * PP + second) * P + 8 * c % P + r;
      Place k{a.w + ((size_t)max(f, 0) * Hkv + kvh) * P + 8 * c % P + r, 0.0f, f >= 0 && key < x.s.L};
      if (k.there && key < x.fresh && a.decay != 0.0f) k.before = *k.p;
      return k;
    };
    Place next{};
    for (int i = 0; i < n; ++i) {
      if ((i & 31) == 0) {
        if (i) {
          look_up(i);
          refill(min(n, i + 32));
        }
        next = place(i);
      }
      const Place mine = next;
      if ((i & 31) < 31 && i + 1 < n) next = place(i + 1);
      const int end = min(n, (i | 31) + 1);
      int f[PP], key0[PP];
      float ks[PP];
      bool some = false, whole = true;
#pragma unroll
      for (int q = 0; q < PP; ++q) {
        const int t = (t0 + i) * PP + q, page = x.page(t);
        f[q] = __shfl_sync(0xffffffffu, ph[q], i & 31);
        ks[q] = __shfl_sync(0xffffffffu, ks_l[q], i & 31);
        key0[q] = f[q] >= 0 ? page * P : kNoKey;
        if (f[q] >= 0 && x.seen(page)) some = true;
        else whole = false;
      }
      float sum[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};  // keys r, r + 8, r + 16, r + 24
      if (some) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bars[warp][used % ST], (used / ST) & 1))) {
          stuck = true;
          break;
        }
        const uint32_t slab = ring + (used % ST) * SLAB;
        bool all = whole;
#pragma unroll
        for (int q = 0; q < PP; ++q)
          all = all && ((key0[q] + P - 1 <= pos_min && key0[q] >= lo_max) || key0[q] + P <= x.sp.pre);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          float s[NT][4];
          k_dot<I8, D, NT>(slab, 16 * mt, lane, bq, s);
          const int q = 16 * mt / P, j0 = key0[q] + (16 * mt) % P + r;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float dot[2] = {s[nt][j], s[nt][2 + j]};
              float v[2];
              q8_scores<true>(dot, v, row[nt][j], ks[q], j0, a.sc, unit, add[nt][j]);
              const bool counts = cf[nt][j] > 0.0f;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float p;
                if constexpr (ENT) {
                  p = fmaxf(v[e], 0.0f);
                  if (a.beta == 2.0f) p *= p;
                  else if (a.beta != 1.0f) p = p > 0.0f ? ex2f(a.beta * __log2f(p)) : 0.0f;
                } else {
                  p = ex2f(v[e]);
                }
                if (!counts || !(all || q8_sees(row[nt][j], j0 + 8 * e, x.sp.pre))) p = 0.0f;
                sum[mt][e] = fmaf(p, cf[nt][j], sum[mt][e]);
              }
            }
        }
        __syncwarp();  // every lane has read the slab
        ++used;
        refill(end);
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sum[mt][e] += __shfl_xor_sync(0xffffffffu, sum[mt][e], 1);
          sum[mt][e] += __shfl_xor_sync(0xffffffffu, sum[mt][e], 2);
        }
      const float got = c & 2 ? (c & 1 ? sum[1][1] : sum[1][0]) : (c & 1 ? sum[0][1] : sum[0][0]);
      if (mine.there) *mine.p = fmaf(mine.before, a.decay, got);
    }
    w += n;
  }
  if (stuck) {  // a copy did not arrive within the bound: flag it, let what was asked for land, stop
    if (lane == 0) {
      raise_flag(a.c.status, ENTMAXKV_DEV_TIMEOUT);
      for (; used < filled; ++used) mbar_wait_bounded(&bars[warp][used % ST], (used / ST) & 1);
    }
    __syncwarp();
  }
}

template <bool I8, int D, int P, int NT, bool ENT>
static cudaError_t weigh_t(const Q8WeighArgs& a, int sms, cudaStream_t st) {
  const int smem = kWeighWarps<NT> * kWeighSlabs<D, NT> * kWeighKeys * D + 1024;
  cudaError_t e = ensure_smem((const void*)weigh_kernel<I8, D, P, NT, ENT>, smem);
  if (e != cudaSuccess) return e;
  CUtensorMap km;
  if ((e = make_q8_map(&km, a.c.k_pool, a.c.nphys, a.c.Hkv, P, D)) != cudaSuccess) return e;
  return launch_k(true, weigh_kernel<I8, D, P, NT, ENT>, dim3(sms), dim3(kWeighWarps<NT> * 32), (size_t)smem, st, a, km);
}
template <bool I8, int D, int P>
static cudaError_t weigh_n(const Q8WeighArgs& a, int sms, cudaStream_t st) {
  if (a.a1 > 0.0f) return weigh_t<I8, D, P, 1, true>(a, sms, st);  // (one row a sequence: a group of at most 8)
  const long long rows = (long long)a.b.max_count * a.c.G;
  if (rows <= 8) return weigh_t<I8, D, P, 1, false>(a, sms, st);
  return rows <= 16 ? weigh_t<I8, D, P, 2, false>(a, sms, st) : weigh_t<I8, D, P, 4, false>(a, sms, st);
}
template <bool I8>
static cudaError_t weigh_d(const Q8WeighArgs& a, int sms, cudaStream_t st) {
  if (a.c.D == 128) return a.c.P == 32 ? weigh_n<I8, 128, 32>(a, sms, st) : weigh_n<I8, 128, 16>(a, sms, st);
  return a.c.P == 32 ? weigh_n<I8, 64, 32>(a, sms, st) : weigh_n<I8, 64, 16>(a, sms, st);
}

cudaError_t launch_weigh_stream(const Q8WeighArgs& a, bool i8, int sms, cudaStream_t st) {
  return i8 ? weigh_d<true>(a, sms, st) : weigh_d<false>(a, sms, st);
}

}  // namespace ekv
