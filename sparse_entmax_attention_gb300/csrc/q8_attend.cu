// q8_attend.cu -- softmax attention of a few rows a sequence over the 8-bit
// paged cache: single tokens of a decode step, drafted tokens, small chunks.
//
//   s_j = scale·ks·(q·code_j) (capped, biased, masked),  o = Σ e^{s_j} vs·code_j / Σ e^{s_j}.
//
// Bound: the pages' bytes. A unit of work is (slot, KV head, row tile) and each
// page of its span; the pages of all units form one line, cut into equal pieces
// for all warps of the device, so sequences of any lengths load it evenly. A
// warp streams its pages through a ring of tensor copies in shared memory:
//   S = K·q^T      m16n8k16 in halves (codes are exact as halves; q is scaled
//                  to exact halves), 16 tokens × 8 rows a tile, fp32 sums;
//   page max m_p, p = 2^{s − m_p} as halves (2^-12), transposed in registers;
//   T = V^T·p      16 dims × 8 rows a tile, fp32 sums of the page alone;
//   acc = acc·2^{m − m'} + T·(vs·2^{m_p − m'}), and the same for Σ p (which
//                  keeps the unrounded p).
// Weights are rounded against their own page's maximum, so many small ones
// behind a large one are not lost. A unit inside one warp's piece is finished
// there; the others leave (m, Σp, acc) pieces which a second kernel joins in
// the order of the line.
#include "q8_tiles.cuh"

namespace ekv {

constexpr int kAttWarps = 8;
constexpr int kAttMaxBlocks = 512;
// Stages of a warp's ring: 24 KB of pages at d = 128, whatever the page size.
template <int P>
constexpr int kAttStages = 96 / P;

static int att_rows(const entmaxkv_config& cfg, int max_count) {
  return (long long)max_count * cfg.group <= 8 ? 8 : 16;
}

// Row tiles and span of a slot; W = its pages on the line.
struct AttSlot {
  Q8Slot s;
  Q8Span sp;
  int nrt;
  long long W;
};
template <int NT>
__device__ __forceinline__ AttSlot att_slot(const Q8AttendArgs& a, int b, uint32_t* st) {
  AttSlot x;
  x.s = q8_slot(a.c, a.b, b, st);
  x.nrt = (x.s.count * a.c.G + 8 * NT - 1) / (8 * NT);
  x.W = 0;
  x.sp = Q8Span{0, 0, 0, 0, 0};
  if (x.s.count > 0) {
    x.sp = q8_span(a.c, a.sc, x.s, b, 0, x.s.count);
    x.W = (long long)x.sp.T * a.c.Hkv * x.nrt;
  }
  return x;
}

// The line's cut: warp w of nw begins at W·w/nw; nw ≤ W, so no piece is empty.
struct AttCut {
  long long W, nw;
  __device__ __forceinline__ long long begin(long long w) const { return W * w / nw; }
  __device__ __forceinline__ long long of(long long at) const { return ((at + 1) * nw - 1) / W; }  // warp that holds `at`
};
__device__ __forceinline__ AttCut att_cut(long long W, int blocks) {
  return AttCut{W, max(1LL, min(W, (long long)blocks * kAttWarps))};
}

// A warp's last piece: the unit that starts at A on the line, T pages long.
struct AttPiece {
  long long A;
  int T, start, kvh, rt, rows;
};

template <bool I8, int D, int P, int NT>
__global__ void __launch_bounds__(kAttWarps * 32, 1)
    attend_kernel(Q8AttendArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  pdl_enter();
  constexpr int NW = kAttWarps, ST = kAttStages<P>, SLAB = P * D, NTH = NW * 32, R = 8 * NT;
  static_assert(R * D * 4 <= ST * 2 * SLAB, "a warp's sums fit its ring");
  extern __shared__ __align__(128) unsigned char dyn_sm[];
  __shared__ uint64_t bars[NW][ST];
  __shared__ long long sh_sum[NW];
  __shared__ long long sh_cum[NW];
  __shared__ int sh_slot[NW];
  __shared__ AttSlot sh_info[NTH];  // the slots, when they are few
  __shared__ AttPiece sh_piece[NW];
  __shared__ float2 sh_ml[NW][R];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring0 = (smem_u32(dyn_sm) + 1023u) & ~1023u;
  const uint32_t ring = ring0 + (uint32_t)warp * ST * 2 * SLAB;
  unsigned char* ring_p = dyn_sm + (ring - smem_u32(dyn_sm));
  if (lane == 0) {
    for (int i = 0; i < ST; ++i) mbar_init(&bars[warp][i], 1);
    mbar_fence_init();
    sh_piece[warp].A = -1;
  }
  // the line: its length, then where each warp's piece begins
  uint32_t* st0 = blockIdx.x == 0 ? a.c.status : nullptr;
  const int n_seqs = a.b.n_seqs;
  const bool few = n_seqs <= NTH;
  long long own = 0;
  for (int b = tid; b < n_seqs; b += NTH) {
    const AttSlot x = att_slot<NT>(a, b, st0);
    own += x.W;
    if (few) sh_info[b] = x;
  }
  long long inc = own;  // inclusive over the block's threads
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) sh_sum[warp] = inc;
  __syncthreads();
  long long W = 0, before = inc - own;
  for (int i = 0; i < NW; ++i) {
    if (i < warp) before += sh_sum[i];
    W += sh_sum[i];
  }
  const AttCut cut = att_cut(W, (int)gridDim.x);
  auto place = [&](int b, long long at, long long n) {  // slot b lies at [at, at + n) of the line
    if (blockIdx.x == 0) a.cum[b] = at;
    for (int i = 0; i < NW; ++i) {
      const long long w = cut.begin((long long)blockIdx.x * NW + i);
      if (at <= w && w < at + n) {
        sh_slot[i] = b;
        sh_cum[i] = at;
      }
    }
  };
  if (few) {
    if (tid < n_seqs) place(tid, before, own);
  } else {
    long long base = 0;
    for (int b0 = 0; b0 < n_seqs; b0 += NTH) {
      const int b = b0 + tid;
      const long long mine = b < n_seqs ? att_slot<NT>(a, b, nullptr).W : 0;
      long long in = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += u;
      }
      __syncthreads();  // the sums of the round before are read
      if (lane == 31) sh_sum[warp] = in;
      __syncthreads();
      long long at = base + in - mine;
      for (int i = 0; i < NW; ++i) {
        if (i < warp) at += sh_sum[i];
        base += sh_sum[i];
      }
      if (b < n_seqs) place(b, at, mine);
    }
  }
  if (blockIdx.x == 0 && tid == 0) a.cum[n_seqs] = W;
  __syncthreads();
  const long long me = (long long)blockIdx.x * NW + warp;
  const long long w_begin = me < cut.nw ? cut.begin(me) : 0, w_end = me < cut.nw ? cut.begin(me + 1) : 0;
  const int G = a.c.G, Hkv = a.c.Hkv;
  const int r = lane >> 2, c = lane & 3;
  const bool general = a.sc.cap > 0.0f || a.sc.slopes;
  int slot = w_begin < w_end ? sh_slot[warp] : 0;
  long long cum = sh_cum[warp];
  long long w = w_begin;
  int filled = 0, used = 0;  // ring fills of this warp, in order
  bool stuck = false;
  while (w < w_end && !stuck) {
    const AttSlot x = few ? sh_info[slot] : att_slot<NT>(a, slot, nullptr);
    if (w >= cum + x.W) {
      cum += x.W;
      ++slot;
      continue;
    }
    const int T = x.sp.T;
    const long long off = w - cum;
    const int u = (int)(off / T), t0 = (int)(off - (long long)u * T);
    const int n = (int)min((long long)(T - t0), w_end - w);
    const int kvh = u / x.nrt, rt = u - kvh * x.nrt;
    const int rows = min(R, x.s.count * G - rt * R);
    // 32 pages' places and scales at once, one a lane; those of the next 32 come in meanwhile
    int ph[2];
    float ks_l[2], vs_l[2];
    auto look_up = [&](int p0, int& f, float& ks, float& vs) {
      f = -1;
      ks = vs = 0.0f;
      if (p0 + lane < n) {
        f = phys_page(a.c.block_table, x.s.seq, x.sp.page(t0 + p0 + lane), a.c.maxp, a.c.nphys, a.c.status);
        if (f >= 0) {
          ks = a.c.k_scale[(size_t)f * Hkv + kvh];
          vs = a.c.v_scale[(size_t)f * Hkv + kvh];
        }
      }
    };
    look_up(0, ph[0], ks_l[0], vs_l[0]);
    ph[1] = -1;
    int ask = 0;  // next page to ask for
    auto refill = [&](int chunk, int end) {
      while (ask < end && filled - used < ST) {
        const int f = __shfl_sync(0xffffffffu, (ask >> 5) == chunk ? ph[0] : ph[1], ask & 31);
        ++ask;
        if (f < 0) continue;
        const int sg = filled % ST;
        if (lane == 0) {
          mbar_expect_tx(&bars[warp][sg], 2 * SLAB);
          tma_load_3d(ring_p + sg * 2 * SLAB, &kmap, 0, kvh * P, f, &bars[warp][sg]);
          tma_load_3d(ring_p + sg * 2 * SLAB + SLAB, &vmap, 0, kvh * P, f, &bars[warp][sg]);
        }
        ++filled;
      }
    };
    refill(0, min(n, 32));  // before the queries are looked at
    // query fragments and row facts
    uint32_t bq[NT][D / 16][2];
    Q8Row row[NT][2];
    int pos_min = 0x7fffffff, lo_max = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rho = rt * R + 8 * nt + r;
      const bool ok = 8 * nt + r < rows;
      const __nv_bfloat16* qp =
          ok ? a.q.p + (long long)(x.s.start + rho / G) * a.q.ts + (long long)(kvh * G + rho % G) * a.q.hs : nullptr;
      float inv;
      q_half_frag<D>(qp, lane, bq[nt], inv);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float f = __shfl_sync(0xffffffffu, inv, (2 * c + j) * 4);
        const int rj = 8 * nt + 2 * c + j, rg = rt * R + rj;
        Q8Row& q = row[nt][j];
        q.cs = f * a.sc.scale * (a.sc.cap > 0.0f ? 1.0f : kLog2e);
        q.slope = 0.0f;
        q.pos = 0;
        q.lo = 0;
        if (rj < rows) {
          const int i = rg / G;
          q.pos = x.s.L - x.s.count + i;
          if (a.sc.window > 0) q.lo = max(0, q.pos - a.sc.window + 1);
          if (a.sc.first_key) q.lo = max(q.lo, a.sc.first_key[x.s.start + i]);
          if (a.sc.slopes) q.slope = a.sc.slopes[kvh * G + rg % G] * kLog2e;
          pos_min = min(pos_min, q.pos);
          lo_max = max(lo_max, q.lo);
        }
      }
    }
    pos_min = __reduce_min_sync(0xffffffffu, pos_min);
    lo_max = __reduce_max_sync(0xffffffffu, lo_max);

    float m[NT][2], l[NT][2], acc[D / 16][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -CUDART_INF_F;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.0f;
    }
    for (int i = 0; i < n; ++i) {
      if ((i & 31) == 0) {
        if (i) {
          ph[0] = ph[1];
          ks_l[0] = ks_l[1];
          vs_l[0] = vs_l[1];
        }
        look_up(i + 32, ph[1], ks_l[1], vs_l[1]);
        refill(i >> 5, min(n, i + 64));
      }
      if (__shfl_sync(0xffffffffu, ph[0], i & 31) < 0) continue;
      const float ks = __shfl_sync(0xffffffffu, ks_l[0], i & 31), vs = __shfl_sync(0xffffffffu, vs_l[0], i & 31);
      const int sg = used % ST;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bars[warp][sg], (used / ST) & 1))) {
        stuck = true;
        break;
      }
      const uint32_t slab = ring + sg * 2 * SLAB;
      const int key0 = x.sp.page(t0 + i) * P;
      const bool whole = (key0 + P - 1 <= pos_min && key0 >= lo_max) || key0 + P <= x.sp.pre;
      if (x.s.L - key0 < P) {  // slots past the sequence's end: any bytes, so that p = 0 meets no NaN
        const int nv = x.s.L - key0;
        for (int e = lane; e < (P - nv) * (D / 16); e += 32)
          *reinterpret_cast<uint4*>(ring_p + sg * 2 * SLAB + SLAB + nv * D + e * 16) = make_uint4(0u, 0u, 0u, 0u);
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
      }
      float s[P / 16][NT][4];
      float pm[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) pm[nt][0] = pm[nt][1] = -CUDART_INF_F;
#pragma unroll
      for (int mt = 0; mt < P / 16; ++mt) {
        k_dot<I8, D, NT>(slab, 16 * mt, lane, bq, s[mt]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = key0 + 16 * mt + r + 8 * (e >> 1);
            float v = q8_score(s[mt][nt][e], row[nt][e & 1], ks, j, a.sc, general, kLog2e);
            if (!whole && !q8_sees(row[nt][e & 1], j, x.sp.pre)) v = -CUDART_INF_F;
            s[mt][nt][e] = v;
            pm[nt][e & 1] = fmaxf(pm[nt][e & 1], v);
          }
      }
      float fv[NT][2], cr[NT][2];
      bool grew = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v = pm[nt][j];
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          const float mn = fmaxf(m[nt][j], v);
          cr[nt][j] = mn > m[nt][j] ? ex2f(m[nt][j] - mn) : 1.0f;  // 0 from -inf
          grew |= mn > m[nt][j];
          fv[nt][j] = v > -CUDART_INF_F ? ex2f(v - mn) : 0.0f;
          m[nt][j] = mn;
          pm[nt][j] = v > -CUDART_INF_F ? v : 0.0f;
        }
      float tmp[D / 16][NT][4];
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) tmp[mt][nt][0] = tmp[mt][nt][1] = tmp[mt][nt][2] = tmp[mt][nt][3] = 0.0f;
      float ls[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) ls[nt][0] = ls[nt][1] = 0.0f;
#pragma unroll
      for (int kt = 0; kt < P / 16; ++kt) {
        uint32_t b[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2f(s[kt][nt][e] - pm[nt][e & 1]);
            ls[nt][e & 1] += p[e];
          }
          const __half2 h0 = __floats2half2_rn(p[0], p[1]), h1 = __floats2half2_rn(p[2], p[3]);
          b[nt][0] = transpose8(*reinterpret_cast<const uint32_t*>(&h0));
          b[nt][1] = transpose8(*reinterpret_cast<const uint32_t*>(&h1));
        }
        v_dot<I8, D, NT>(slab + SLAB, 16 * kt, lane, b, tmp);
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          l[nt][0] *= cr[nt][0];
          l[nt][1] *= cr[nt][1];
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][nt][e] *= cr[nt][e & 1];
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        l[nt][0] = fmaf(ls[nt][0], fv[nt][0], l[nt][0]);
        l[nt][1] = fmaf(ls[nt][1], fv[nt][1], l[nt][1]);
        const float f0 = fv[nt][0] * vs, f1 = fv[nt][1] * vs;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[mt][nt][e] = fmaf(tmp[mt][nt][e], e & 1 ? f1 : f0, acc[mt][nt][e]);
      }
      __syncwarp();  // every lane has read the stage
      ++used;
      refill(i >> 5, min(n, ((i >> 5) + 2) * 32));
    }
    if (stuck) break;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
      }
    const bool last = w + n == w_end;
    if (n == T) {  // the whole unit
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int rj = 8 * nt + 2 * c + j;
          if (rj >= rows) continue;
          const int rg = rt * R + rj;
          const long long tok = x.s.start + rg / G;
          const int h = kvh * G + rg % G;
          const float inv = att_inv(l[nt][j]);
          __nv_bfloat16* o = a.out.p + tok * a.out.ts + (long long)h * a.out.hs;
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt)
            *reinterpret_cast<uint32_t*>(o + 16 * mt + 2 * r) = bf2_rn(acc[mt][nt][j] * inv, acc[mt][nt][2 + j] * inv);
          if (a.tau && r == 0) a.tau[tok * Hkv * G + h] = att_lse(m[nt][j], l[nt][j]);
        }
    } else {
      // a piece that this warp goes on behind leaves for the joining kernel; the last one waits for its
      // neighbours' in the ring, which is done with
      float* to = last ? reinterpret_cast<float*>(ring_p) : a.part_o + (size_t)me * 2 * R * D;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int rj = 8 * nt + 2 * c + j;
          if (rj >= rows) continue;
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt)
            *reinterpret_cast<float2*>(to + rj * D + 16 * mt + 2 * r) = make_float2(acc[mt][nt][j], acc[mt][nt][2 + j]);
          if (r == 0) {
            if (last) sh_ml[warp][rj] = make_float2(m[nt][j], l[nt][j]);
            else reinterpret_cast<float2*>(a.part_ml)[(size_t)me * 2 * R + rj] = make_float2(m[nt][j], l[nt][j]);
          }
        }
      if (last && lane == 0) sh_piece[warp] = AttPiece{w - t0, T, x.s.start, kvh, rt, rows};
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
  __syncthreads();
  // the warps' last pieces: neighbours of one unit are joined here
  for (int i0 = 0, i1; i0 < NW; i0 = i1) {
    i1 = i0 + 1;
    const AttPiece x = sh_piece[i0];
    if (x.A < 0) continue;
    while (i1 < NW && sh_piece[i1].A == x.A) ++i1;
    const long long first = (long long)blockIdx.x * NW + i0;
    const bool all = cut.begin(first) <= x.A && cut.begin((long long)blockIdx.x * NW + i1) == x.A + x.T;
    for (int e = tid; e < x.rows * D; e += NTH) {
      const int rj = e / D;
      float M = -CUDART_INF_F;
      for (int i = i0; i < i1; ++i) M = fmaxf(M, sh_ml[i][rj].x);
      float l = 0.0f, o = 0.0f;
      for (int i = i0; i < i1; ++i) {
        const float2 ml = sh_ml[i][rj];
        const float f = ml.x > -CUDART_INF_F ? ex2f(ml.x - M) : 0.0f;
        l = fmaf(f, ml.y, l);
        o = fmaf(f, reinterpret_cast<const float*>(dyn_sm + (ring0 - smem_u32(dyn_sm)) + i * ST * 2 * SLAB)[e], o);
      }
      if (all) {
        const int rg = x.rt * R + rj;
        const long long tok = x.start + rg / G;
        const int h = x.kvh * G + rg % G;
        a.out.p[tok * a.out.ts + (long long)h * a.out.hs + e % D] = __float2bfloat16_rn(o * att_inv(l));
        if (a.tau && e % D == 0) a.tau[tok * Hkv * G + h] = att_lse(M, l);
      } else {
        const size_t piece = (size_t)first * 2 + 1;
        a.part_o[piece * R * D + e] = o;
        if (e % D == 0) reinterpret_cast<float2*>(a.part_ml)[piece * R + rj] = make_float2(M, l);
      }
    }
  }
}

// Joins the pieces of units that several blocks hold, and answers rows that see
// no page at all. A unit's pieces, in the order of the line: one a block from
// its first warp on (left by the block's first warp of the unit), and where its
// last warp goes on behind it, that warp's own. Block (KV head · row tile ·
// row, slot), a thread a dimension.
template <int D, int NT>
__global__ void __launch_bounds__(D) attend_join_kernel(Q8AttendArgs a, int nrt_max) {
  pdl_enter();
  constexpr int R = 8 * NT, NW = kAttWarps;
  const int b = blockIdx.y, rj = blockIdx.x % R, rt = blockIdx.x / R % nrt_max, kvh = blockIdx.x / R / nrt_max;
  const AttSlot x = att_slot<NT>(a, b, nullptr);
  const int G = a.c.G;
  if (rt >= x.nrt || rj >= x.s.count * G - rt * R) return;
  const long long W = a.cum[a.b.n_seqs];
  const AttCut cut = att_cut(W, a.blocks);
  const int T = x.sp.T;
  const long long A = a.cum[b] + ((long long)kvh * x.nrt + rt) * T, B = A + T;
  float M = -CUDART_INF_F, l = 0.0f, o = 0.0f;
  if (T > 0) {
    const long long w0 = cut.of(A), w1 = cut.of(B - 1);
    const bool tail = cut.begin(w1 + 1) > B;  // the last warp goes on: its piece lies apart
    if (w0 == w1 || (!tail && w0 / NW == w1 / NW)) return;  // finished by that warp or block
    const long long c0 = w0 / NW, c1 = (tail ? w1 - 1 : w1) / NW;
    const int n = (int)(c1 - c0 + 1) + (tail ? 1 : 0);
    auto piece = [&](int i) -> size_t {
      if (c0 + i > c1) return (size_t)w1 * 2;
      return (size_t)(i ? (c0 + i) * NW : w0) * 2 + 1;
    };
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
#pragma unroll 4
    for (int i = 0; i < n; ++i) M = fmaxf(M, ml[piece(i) * R + rj].x);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float2 v = ml[piece(i) * R + rj];
      const float f = v.x > -CUDART_INF_F ? ex2f(v.x - M) : 0.0f;
      l = fmaf(f, v.y, l);
      o = fmaf(f, a.part_o[(piece(i) * R + rj) * D + threadIdx.x], o);
    }
  }
  const int rg = rt * R + rj;
  const long long tok = x.s.start + rg / G;
  const int h = kvh * G + rg % G;
  a.out.p[tok * a.out.ts + (long long)h * a.out.hs + threadIdx.x] = __float2bfloat16_rn(o * att_inv(l));
  if (a.tau && threadIdx.x == 0) a.tau[tok * a.c.Hkv * G + h] = att_lse(M, l);
}

cudaError_t make_q8_map(CUtensorMap* map, const void* pool, int nphys, int Hkv, int P, int D) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hkv * P, (cuuint64_t)nphys};
  const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)Hkv * P * D};
  const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)P, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pool), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE,
                         D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

static size_t up256z(size_t x) { return (x + 255) & ~(size_t)255; }

size_t attend_softmax_bytes(const entmaxkv_config& cfg, int n_seqs, int max_count) {
  const size_t pieces = (size_t)kAttMaxBlocks * kAttWarps * 2 * att_rows(cfg, max_count);
  return up256z((size_t)(n_seqs + 1) * 8) + up256z(pieces * cfg.head_dim * 4) + up256z(pieces * 8);
}

template <bool I8, int D, int P, int NT>
static cudaError_t attend_t(Q8AttendArgs& a, void* ws, int sms, cudaStream_t st) {
  const int smem = kAttWarps * kAttStages<P> * 2 * P * D + 1024;
  cudaError_t e = ensure_smem((const void*)attend_kernel<I8, D, P, NT>, smem);
  if (e != cudaSuccess) return e;
  CUtensorMap km, vm;
  if ((e = make_q8_map(&km, a.c.k_pool, a.c.nphys, a.c.Hkv, P, D)) != cudaSuccess) return e;
  if ((e = make_q8_map(&vm, a.c.v_pool, a.c.nphys, a.c.Hkv, P, D)) != cudaSuccess) return e;
  a.blocks = min(sms, kAttMaxBlocks);
  char* p = static_cast<char*>(ws);
  const size_t pieces = (size_t)kAttMaxBlocks * kAttWarps * 2 * 8 * NT;
  a.cum = reinterpret_cast<long long*>(p);
  p += up256z((size_t)(a.b.n_seqs + 1) * 8);
  a.part_o = reinterpret_cast<float*>(p);
  p += up256z(pieces * D * 4);
  a.part_ml = reinterpret_cast<float*>(p);
  e = launch_k(false, attend_kernel<I8, D, P, NT>, dim3(a.blocks), dim3(kAttWarps * 32), (size_t)smem, st, a, km, vm);
  if (e != cudaSuccess) return e;
  const int nrt = (int)(((long long)a.b.max_count * a.c.G + 8 * NT - 1) / (8 * NT));
  return launch_k(false, attend_join_kernel<D, NT>, dim3(nrt * 8 * NT * a.c.Hkv, a.b.n_seqs), dim3(D), 0,
                  st, a, nrt);
}

template <bool I8, int D, int P>
static cudaError_t attend_n(Q8AttendArgs& a, void* ws, int sms, cudaStream_t st) {
  return (long long)a.b.max_count * a.c.G <= 8 ? attend_t<I8, D, P, 1>(a, ws, sms, st)
                                               : attend_t<I8, D, P, 2>(a, ws, sms, st);
}
template <bool I8>
static cudaError_t attend_d(Q8AttendArgs& a, void* ws, int sms, cudaStream_t st) {
  if (a.c.D == 128)
    return a.c.P == 32 ? attend_n<I8, 128, 32>(a, ws, sms, st) : attend_n<I8, 128, 16>(a, ws, sms, st);
  return a.c.P == 32 ? attend_n<I8, 64, 32>(a, ws, sms, st) : attend_n<I8, 64, 16>(a, ws, sms, st);
}

cudaError_t launch_attend_softmax(Q8AttendArgs a, bool i8, void* ws, int sms, cudaStream_t st) {
  return i8 ? attend_d<true>(a, ws, sms, st) : attend_d<false>(a, ws, sms, st);
}

}  // namespace ekv
