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
//                  to exact halves), 16 tokens × 8 rows a product, fp32 sums;
//   t = S·ks·scale·log2 e (capped, biased, masked) + log2 vs
//   w = 2^{t − M + 8} as halves (off by 2^-11, an eighth of the bf16 output's
//                  rounding; a second half would double the products), transposed in registers, M a bound of
//                  the row's maximum that moves when a t passes it by 6 (a vote
//                  a tile; the maximum itself is only formed then): w ≤ 2^14, and
//                  weights down to 2^-32 of the largest survive the rounding;
//   acc += V^T·w   16 dims × 8 rows a product, fp32; Σp is Σ over pages of
//                  (Σ w)/vs, of unrounded w.
// A tile is 32 keys: one page, or two of 16. A unit inside one warp's piece is
// finished there, neighbouring warps of a block join theirs in shared memory,
// and the rest leaves (M, Σp, acc) pieces which a second kernel joins in the
// order of the line.
//
// Measured (graph replays, inputs in turn): 16 sequences of 4-65k tokens, 8 KV heads of 4 query
// heads, d = 128, e4m3, capped, with slopes (756 MB): 135 us, 5.6 TB/s,
// 0.83 of the measured copy rate. Time over bytes is 6.3 TB/s and 8-10 us for
// start, block join and join kernel, which is what a single sequence of 32k
// tokens (67 MB) feels: 27.5 us (23.3 where L2 holds them). In a capture (789 MB, 131 us) the pipes wait
// for nothing in particular: ALU 48% (codes to halves), IPC 2.2.
#include "q8_tiles.cuh"

namespace ekv {

// Warps of a block, and K or V slabs (32·D bytes) of a warp's ring, 196 KB in all:
// 16 warps fit 128 registers with one tile of 8 rows (the ragged batch above: 136
// us, against 199 with 8 of them on whole pages), or with two at d = 64; at d = 128
// two tiles need twice as many.
template <int D, int NT>
constexpr int kAttWarps = NT == 2 && D == 128 ? 8 : 16;
template <int D, int NT>
constexpr int kAttSlabs = 192 * 1024 / (kAttWarps<D, NT> * 32 * D);
constexpr int kAttMaxBlocks = 256;
constexpr int kAttKeys = 32;

// Row tiles (8·NT rows each), tiles of keys and span of a slot; W = its tiles on
// the line, the row tiles of a KV head one behind the other.
struct AttSlot {
  Q8Slot s;
  Q8Span sp;
  int nrt, T;
  long long W;
};
template <int NT>
__device__ __forceinline__ AttSlot att_slot(const Q8AttendArgs& a, int b, uint32_t* st) {
  AttSlot x;
  x.s = q8_slot(a.c, a.b, b, st);
  x.nrt = (int)((uint32_t)(x.s.count * a.c.G + 8 * NT - 1) / (uint32_t)(8 * NT));
  x.W = 0;
  x.T = 0;
  x.sp = Q8Span{0, 0, 0, 0, 0};
  if (x.s.count > 0) {
    x.sp = q8_span(a.c, a.sc, x.s, b, 0, x.s.count);
    x.T = (x.sp.T * a.c.P + kAttKeys - 1) / kAttKeys;
    x.W = (long long)x.T * a.c.Hkv * x.nrt;
  }
  return x;
}

// A warp's last piece: the unit that starts at A on the line, T pages long.
struct AttPiece {
  long long A;
  int T, start, kvh, row0, rows;
};

template <bool I8, int D, int P, int NT>
__global__ void __launch_bounds__(kAttWarps<D, NT> * 32, 1)
    attend_kernel(Q8AttendArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  pdl_enter();
  constexpr int NW = kAttWarps<D, NT>, ST = kAttSlabs<D, NT>, SLAB = kAttKeys * D, NTH = NW * 32, R = 8 * NT;
  constexpr int PP = kAttKeys / P;  // pages a tile
  static_assert(R * D * 4 <= ST * SLAB, "a warp's sums fit its ring");
  extern __shared__ __align__(128) unsigned char dyn_sm[];
  __shared__ uint64_t bars[NW][ST];
  __shared__ LineSmem<NW> sh_line;
  constexpr int kFew = 256;
  __shared__ AttSlot sh_info[kFew];  // the slots, when they are few
  __shared__ AttPiece sh_piece[NW];
  __shared__ float2 sh_ml[NW][R];
  __shared__ float sh_f[NW][R];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring0 = (smem_u32(dyn_sm) + 1023u) & ~1023u;
  const uint32_t ring = ring0 + (uint32_t)warp * ST * SLAB;
  unsigned char* ring_p = dyn_sm + (ring - smem_u32(dyn_sm));
  if (lane == 0) {
    for (int i = 0; i < ST; ++i) mbar_init(&bars[warp][i], 1);
    mbar_fence_init();
    sh_piece[warp].A = -1;
  }
  if (tid == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  const int n_seqs = a.b.n_seqs;
  const bool few = n_seqs <= kFew;
  const LinePlace at = line_place<NW>(
      n_seqs, a.c.status, sh_line,
      [&](int b, uint32_t* st) {
        const AttSlot x = att_slot<NT>(a, b, st);
        if (few) sh_info[b] = x;
        return x.W;
      },
      [&](int b, long long where) {
        a.cum[b] = where;
        if (b < n_seqs) reinterpret_cast<AttSlot*>(a.slots)[b] = few ? sh_info[b] : att_slot<NT>(a, b, nullptr);
      });
  const LineCut cut = at.cut;
  const long long me = (long long)blockIdx.x * NW + warp;
  const long long w_begin = at.begin, w_end = at.end;
  const int G = a.c.G, Hkv = a.c.Hkv;
  const int r = lane >> 2, c = lane & 3;
  int slot = at.slot;
  long long cum = at.cum;
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
    const int T = x.T;
    const long long off = w - cum;
    const int unit = (int)div_line(off, T), t0 = (int)(off - (long long)unit * T);
    const int n = (int)min((long long)(T - t0), w_end - w);
    const int kvh = (int)((uint32_t)unit / (uint32_t)x.nrt), row0 = (unit - kvh * x.nrt) * R;
    const int rows = min(R, x.s.count * G - row0);
    // 32 tiles' places and scales at once, a tile a lane
    int ph[PP];
    float ks_l[PP], vs_l[PP];
    auto look_up = [&](int p0) {
#pragma unroll
      for (int q = 0; q < PP; ++q) {
        const int t = (t0 + n - 1 - p0 - lane) * PP + q;  // nearest keys first: a distance bias sets the bound at once
        ph[q] = -1;
        ks_l[q] = 0.0f;
        vs_l[q] = 1.0f;
        if (p0 + lane < n && t < x.sp.T) {
          ph[q] = phys_page(a.c.block_table, x.s.seq, x.sp.page(t), a.c.maxp, a.c.nphys, a.c.status);
          if (ph[q] >= 0) {
            ks_l[q] = a.c.k_scale[(size_t)ph[q] * Hkv + kvh];
            vs_l[q] = a.c.v_scale[(size_t)ph[q] * Hkv + kvh];
          }
        }
      }
    };
    int ask = 0;  // next slab to ask for: K and V of a tile in turn
    auto refill = [&](int end) {
      while (ask < 2 * end && filled - used < ST) {
        int f[PP], there = 0;
#pragma unroll
        for (int q = 0; q < PP; ++q) {
          f[q] = __shfl_sync(0xffffffffu, ph[q], (ask >> 1) & 31);
          there += f[q] >= 0;
        }
        const int side = ask & 1;
        ++ask;
        if (!there) continue;
        const int sg = filled % ST;
        if (lane == 0) {
          mbar_expect_tx(&bars[warp][sg], (uint32_t)(there * P * D));
#pragma unroll
          for (int q = 0; q < PP; ++q)
            if (f[q] >= 0)
              tma_load_3d(ring_p + sg * SLAB + q * P * D, side ? &vmap : &kmap, 0, kvh * P, f[q], &bars[warp][sg]);
        }
        ++filled;
      }
    };
    // the queries come in beside the pages' places; the first pages are asked for before they are looked at
    uint4 qw[NT][D / 32];
    uint32_t bq[NT][D / 16][2];
    Q8Row row[NT][2];
    int pos_min = 0x7fffffff, lo_max = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t rho = row0 + 8 * nt + r, tok = rho / (uint32_t)G;
      q_load<D>(8 * nt + r < rows ? a.q.p + (long long)(x.s.start + (int)tok) * a.q.ts +
                                      (long long)(kvh * G + (int)(rho - tok * G)) * a.q.hs
                                : nullptr,
                lane, qw[nt]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t rj = row0 + 8 * nt + 2 * c + j, i = rj / (uint32_t)G;
        Q8Row& q = row[nt][j];
        q.slope = 0.0f;
        q.pos = 0;
        q.lo = 0;
        if (8 * nt + 2 * c + j < rows) {
          q.pos = x.s.L - x.s.count + (int)i;
          if (a.sc.window > 0) q.lo = max(0, q.pos - a.sc.window + 1);
          if (a.sc.first_key) q.lo = max(q.lo, a.sc.first_key[x.s.start + (int)i]);
          if (a.sc.slopes) q.slope = a.sc.slopes[kvh * G + (int)(rj - i * G)] * kLog2e;
          pos_min = min(pos_min, q.pos);
          lo_max = max(lo_max, q.lo);
        }
      }
    }
    look_up(0);
    refill(min(n, 32));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float inv;
      q_half_frag<D>(qw[nt], bq[nt], inv);
#pragma unroll
      for (int j = 0; j < 2; ++j) row[nt][j].cs = q8_row_scale(__shfl_sync(0xffffffffu, inv, (2 * c + j) * 4), a.sc, kLog2e);
    }
    pos_min = __reduce_min_sync(0xffffffffu, pos_min);
    lo_max = __reduce_max_sync(0xffffffffu, lo_max);

    float m[NT][2], l[NT][2], acc[D / 16][NT][4];  // M, Σp, Σ w·code
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -CUDART_INF_F;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.0f;
    }
    for (int i = 0; i < n; ++i) {
      if ((i & 31) == 0 && i) {
        look_up(i);
        refill(min(n, i + 32));
      }
      const int end = min(n, (i | 31) + 1);
      int f[PP], key0[PP];
      float ks[PP], vs[PP];
      bool some = false, whole = true;
#pragma unroll
      for (int q = 0; q < PP; ++q) {
        f[q] = __shfl_sync(0xffffffffu, ph[q], i & 31);
        ks[q] = __shfl_sync(0xffffffffu, ks_l[q], i & 31);
        vs[q] = fmaxf(__shfl_sync(0xffffffffu, vs_l[q], i & 31), 0x1p-100f);
        key0[q] = f[q] >= 0 ? x.sp.page((t0 + n - 1 - i) * PP + q) * P : kNoKey;
        some |= f[q] >= 0;
        whole &= (key0[q] + P - 1 <= pos_min && key0[q] >= lo_max) || key0[q] + P <= x.sp.pre;
      }
      if (!some) continue;
      auto arrived = [&]() -> bool {
        return __all_sync(0xffffffffu, mbar_wait_bounded(&bars[warp][used % ST], (used / ST) & 1));
      };
      if (!arrived()) {
        stuck = true;
        break;
      }
      uint32_t slab = ring + (used % ST) * SLAB;
      float s[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        k_dot<I8, D, NT>(slab, 16 * mt, lane, bq, s[mt]);
        const int q = 16 * mt / P, j0 = key0[q] + (16 * mt) % P + r;
        const float lv = __log2f(vs[q]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float dot[2] = {s[mt][nt][j], s[mt][nt][2 + j]};
            float v[2];
            q8_scores(dot, v, row[nt][j], ks[q], j0, a.sc, kLog2e, lv);
            if (!whole) {
              if (!q8_sees(row[nt][j], j0, x.sp.pre)) v[0] = -CUDART_INF_F;
              if (!q8_sees(row[nt][j], j0 + 8, x.sp.pre)) v[1] = -CUDART_INF_F;
            }
            s[mt][nt][j] = v[0];
            s[mt][nt][2 + j] = v[1];
          }
      }
      __syncwarp();  // every lane has read the K slab
      ++used;
      refill(end);
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          over |= fmaxf(max3(s[0][nt][j], s[0][nt][2 + j], s[1][nt][j]), s[1][nt][2 + j]) > m[nt][j] + kSlack;
      if (__any_sync(0xffffffffu, over)) {  // some bound moves
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float v = fmaxf(fmaxf(s[0][nt][j], s[0][nt][2 + j]), fmaxf(s[1][nt][j], s[1][nt][2 + j]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            if (v > m[nt][j] + kSlack) {
              const float cr = ex2f(m[nt][j] - v);  // 0 from -inf
              m[nt][j] = v;
              l[nt][j] *= cr;
#pragma unroll
              for (int mt = 0; mt < D / 16; ++mt) {
                acc[mt][nt][j] *= cr;
                acc[mt][nt][2 + j] *= cr;
              }
            }
          }
      }
      if (!arrived()) {
        stuck = true;
        break;
      }
      slab = ring + (used % ST) * SLAB;
      if (!whole) {  // slots past the sequence's end, or of no page: any bytes, so that w = 0 meets no NaN
        bool wrote = false;
#pragma unroll
        for (int q = 0; q < PP; ++q) {
          const int nv = max(0, min(P, x.s.L - key0[q]));
          if (nv == P) continue;
          for (int e = lane; e < (P - nv) * (D / 16); e += 32)
            *reinterpret_cast<uint4*>(ring_p + (used % ST) * SLAB + (q * P + nv) * D + e * 16) = make_uint4(0u, 0u, 0u, 0u);
          wrote = true;
        }
        if (wrote) {
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          __syncwarp();
        }
      }
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        uint32_t b[NT][2];
        const float ivs = __fdividef(1.0f, vs[16 * kt / P]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[e] = ex2f(s[kt][nt][e] + (m[nt][e & 1] > -CUDART_INF_F ? kLift - m[nt][e & 1] : 0.0f));
          l[nt][0] = fmaf(p[0] + p[2], ivs, l[nt][0]);
          l[nt][1] = fmaf(p[1] + p[3], ivs, l[nt][1]);
          const __half2 h0 = __floats2half2_rn(p[0], p[1]), h1 = __floats2half2_rn(p[2], p[3]);
          b[nt][0] = transpose8(*reinterpret_cast<const uint32_t*>(&h0));
          b[nt][1] = transpose8(*reinterpret_cast<const uint32_t*>(&h1));
        }
        v_dot<I8, D, NT>(slab, 16 * kt, lane, b, acc);
      }
      __syncwarp();  // every lane has read the V slab
      ++used;
      refill(end);
    }
    if (stuck) break;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
        m[nt][j] -= kLift;
      }
    const bool last = w + n == w_end;
    if (n == T) {  // the whole unit
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int rj = 8 * nt + 2 * c + j;
          if (rj >= rows) continue;
          const int i = (int)((uint32_t)(row0 + rj) / (uint32_t)G), h = kvh * G + row0 + rj - i * G;
          const long long tok = x.s.start + i;
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
      if (last && lane == 0) sh_piece[warp] = AttPiece{w - t0, T, x.s.start, kvh, row0, rows};
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
  // the warps' last pieces: neighbours of one unit are joined here. First each row's maximum and the pieces' factors
  // (a lane a piece, its row's other pieces by shuffles)
  static_assert(NW * R <= NTH && 32 % NW == 0, "NW lanes a row, 32/NW rows a warp");
  if (tid < NW * R) {
    const int i = tid % NW, rj = tid / NW;
    const AttPiece& x = sh_piece[i];
    const bool in = x.A >= 0 && rj < x.rows;
    const int unit = in ? (int)x.A : -1;
    const float2 v = in ? sh_ml[i][rj] : make_float2(-CUDART_INF_F, 0.0f);
    float M = v.x;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const int u = __shfl_sync(0xffffffffu, unit, k, NW);
      const float y = __shfl_sync(0xffffffffu, v.x, k, NW);
      if (u == unit) M = fmaxf(M, y);
    }
    const float f = v.x > -CUDART_INF_F ? ex2f(v.x - M) : 0.0f;
    float l = 0.0f;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const int u = __shfl_sync(0xffffffffu, unit, k, NW);
      const float y = __shfl_sync(0xffffffffu, f * v.y, k, NW);
      if (u == unit) l += y;
    }
    sh_f[i][rj] = f;
    sh_ml[i][rj] = make_float2(M, l);
  }
  __syncthreads();
  for (int i0 = 0, i1; i0 < NW; i0 = i1) {
    i1 = i0 + 1;
    const AttPiece x = sh_piece[i0];
    if (x.A < 0) continue;
    while (i1 < NW && sh_piece[i1].A == x.A) ++i1;
    const long long first = (long long)blockIdx.x * NW + i0;
    const bool all = cut.begin(first) <= x.A && cut.begin((long long)blockIdx.x * NW + i1) == x.A + x.T;
    const float* ring_f = reinterpret_cast<const float*>(dyn_sm + (ring0 - smem_u32(dyn_sm)));
    for (int e = tid; e < x.rows * D; e += NTH) {
      const int rj = e / D;
      float o = 0.0f;
#pragma unroll 4
      for (int i = i0; i < i1; ++i) o = fmaf(sh_f[i][rj], ring_f[i * (ST * SLAB / 4) + e], o);
      const float M = sh_ml[i0][rj].x, l = sh_ml[i0][rj].y;
      if (all) {
        const int i = (int)((uint32_t)(x.row0 + rj) / (uint32_t)G), h = x.kvh * G + x.row0 + rj - i * G;
        const long long tok = x.start + i;
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
// last warp goes on behind it, that warp's own. Block (KV head · row tile · row,
// slot), a thread a dimension.
template <int D, int NT>
__global__ void __launch_bounds__(D) attend_join_kernel(Q8AttendArgs a, int nrt_max) {
  pdl_enter();
  constexpr int R = 8 * NT, NW = kAttWarps<D, NT>;
  const int b = blockIdx.y, rj = blockIdx.x % R, unit = blockIdx.x / R, kvh = unit / nrt_max, rt = unit - kvh * nrt_max;
  const AttSlot x = reinterpret_cast<const AttSlot*>(a.slots)[b];
  const long long W = a.cum[a.b.n_seqs], at = a.cum[b];
  const int G = a.c.G;
  if (rt >= x.nrt || rt * R + rj >= x.s.count * G) return;
  const LineCut cut = line_cut(W, a.blocks, NW);
  const int T = x.T;
  const long long A = at + ((long long)kvh * x.nrt + rt) * T, B = A + T;
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
    for (int i0 = 0; i0 < n; i0 += 8) {  // eight pieces' loads in flight
      float2 v[8];
      float p[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = make_float2(-CUDART_INF_F, 0.0f);
        p[k] = 0.0f;
        if (i0 + k < n) {
          const size_t at8 = piece(i0 + k) * R + rj;
          v[k] = ml[at8];
          p[k] = a.part_o[at8 * D + threadIdx.x];
        }
      }
      float m = M;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = fmaxf(m, v[k].x);
      const float old = M > -CUDART_INF_F ? ex2f(M - m) : 0.0f;
      l *= old;
      o *= old;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float f = v[k].x > -CUDART_INF_F ? ex2f(v[k].x - m) : 0.0f;
        l = fmaf(f, v[k].y, l);
        o = fmaf(f, p[k], o);
      }
      M = m;
    }
  }
  const int i = (int)((uint32_t)(rt * R + rj) / (uint32_t)G), h = kvh * G + rt * R + rj - i * G;
  const long long tok = x.s.start + i;
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

size_t attend_softmax_bytes(const entmaxkv_config& cfg, int n_seqs) {
  const size_t pieces = (size_t)kAttMaxBlocks * 16 * 2 * (cfg.head_dim == 64 ? 16 : 8);  // 16 warps of a tile or two
  return up256z((size_t)(n_seqs + 1) * 8) + up256z((size_t)n_seqs * sizeof(AttSlot)) +
         up256z(pieces * cfg.head_dim * 4) + up256z(pieces * 8);
}

template <bool I8, int D, int P, int NT>
static cudaError_t attend_t(Q8AttendArgs& a, void* ws, int sms, cudaStream_t st) {
  const int smem = kAttWarps<D, NT> * kAttSlabs<D, NT> * kAttKeys * D + 1024;
  cudaError_t e = ensure_smem((const void*)attend_kernel<I8, D, P, NT>, smem);
  if (e != cudaSuccess) return e;
  CUtensorMap km, vm;
  if ((e = make_q8_map(&km, a.c.k_pool, a.c.nphys, a.c.Hkv, P, D)) != cudaSuccess) return e;
  if ((e = make_q8_map(&vm, a.c.v_pool, a.c.nphys, a.c.Hkv, P, D)) != cudaSuccess) return e;
  a.blocks = min(sms, kAttMaxBlocks);
  char* p = static_cast<char*>(ws);
  const size_t pieces = (size_t)kAttMaxBlocks * kAttWarps<D, NT> * 2 * 8 * NT;
  a.cum = reinterpret_cast<long long*>(p);
  p += up256z((size_t)(a.b.n_seqs + 1) * 8);
  a.slots = p;
  p += up256z((size_t)a.b.n_seqs * sizeof(AttSlot));
  a.part_o = reinterpret_cast<float*>(p);
  p += up256z(pieces * D * 4);
  a.part_ml = reinterpret_cast<float*>(p);
  e = launch_k(false, attend_kernel<I8, D, P, NT>, dim3(a.blocks), dim3(kAttWarps<D, NT> * 32), (size_t)smem, st, a, km, vm);
  if (e != cudaSuccess) return e;
  const int nrt = (int)(((long long)a.b.max_count * a.c.G + 8 * NT - 1) / (8 * NT));
  return launch_k(true, attend_join_kernel<D, NT>, dim3(8 * NT * nrt * a.c.Hkv, a.b.n_seqs), dim3(D), 0, st, a, nrt);
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
