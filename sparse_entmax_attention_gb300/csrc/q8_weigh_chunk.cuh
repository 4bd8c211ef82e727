// q8_weigh_chunk.cuh -- the weight that many rows a sequence give to the keys of
// the 8-bit paged cache, on the fifth-generation tensor cores.
//
//   w_j ← decay·w_j + Σ over rows of 2^{t_j},  t_j = s_j·log2 e − tau·log2 e + log2 coef
//
// (s_j capped, biased, masked). A block holds 256 keys of a (slot, KV head) and
// lets the rows pass, 128 (token, head of the group) at a time:
//   S^T = K·Q^T   two products of 128 keys × 128 rows, codes and queries as halves,
//                 fp32 sums in tensor memory, keys along the lanes: a thread has
//                 one key, and its sum over the rows needs no other;
//   Σ 2^t         a key's scale is the thread's, what belongs to a row comes as a
//                 broadcast from shared memory: an FMA, an exponential and an
//                 addition a pair, the first and the last on two rows at once.
//
// Codes are exact in halves, at a quarter to a half of the instructions of bf16 (a tile of
// keys took as much of the issue as a tile of rows does). Queries are brought by a power of
// two to [2^14, 2^15) at their tile's largest: a value down to 2^-29 of that stays exact,
// and what smaller ones lose is at most 2^-39 of it, in the score, of which a weight is the
// exponential, far less than the fp32 sum's own rounding of the largest row.
//
// A first pass lays the rows out as the products and the sums want them: tiles of
// 128 queries in the operand's swizzled order, and what belongs to a row. (Copied
// row by row from where they lie, a tile of rows took 1600 cycles to come in, more
// than the products with it.)
//
// Warps: 16 of sums (two threads a key, one for each 64 rows of a tile: four warps a
// scheduler hide one another's waits); 8 that bring the keys (the next 256 wait as
// codes in registers until the products with the present ones are done); 2 that
// issue the products, one for each 128 keys; 1 that asks for the rows, two tiles
// ahead; 1 that looks up the segments ahead of them all. Segments (key tile, share of
// the rows) go round the blocks in turns; rows are shared out only where there are
// few key tiles, and the block that finishes a tile last adds its shares in their
// order. (Segments handed out as blocks are done with the last: no faster.)
//
// Bound: latency and issue of the sums. A tile of rows (256 keys × 128 rows) takes
// them about 1700 cycles; its exponentials alone are 1024 (32 a clock and
// multiprocessor), its products 1024, and the two meet in shared memory, where the
// operands and the rows' facts are read. Measured, int8, 8 KV heads of 4 query heads,
// d = 128: 2048 rows on 30001 keys before them (0.52 TFLOP) 408 us with listing and
// packing (15 us), 1275 TFLOP/s, 0.65 of the measured bf16 burst; in a capture
// (10240 keys) exponentials 55%, tensor pipe 54%, IPC 2.3; the last 64 rows of six prompts of 500-32000, e4m3, 63 us.
// Kept aside, measured: two
// warps of sums a scheduler 543 us; one key tile in shared memory (four stages of rows)
// 463; keys in tensor memory and tiles of 96 rows 435-463, with the last rows of six
// prompts at 77 us instead of 64; single fp32 operations in place of pairs 482.
#pragma once

#include "q8_chunk.cuh"

namespace ekv {

constexpr int kWcThreads = 896;
constexpr int kWcKeys = 256, kWcRows = 128;
// Stages of the rows, and of their facts, which the sums read longer: the facts of unit u are asked for when the
// products of u − kWcQ are done, so the sums of u − kWcQ − 2 are.
constexpr int kWcQ = 2, kWcMeta = kWcQ + 2, kWcSegs = 5, kWcK = 2;
constexpr int kWcMaxBlocks = 256;
constexpr int kWcTurns = 3;  // segments a block should get at least (12, 6, 3: 109, 97, 88 us for 1024 rows on 8001 keys)

struct __align__(16) WcSlot {
  int seq, L, start, count;        // Q8Slot
  int pre, npre, wfirst, npages;   // Q8Span
  int lnpre, lwfirst, fresh, T;    // pages on the line, first fresh key, key tiles
  int nrt, rt0, nsplit, pad;       // row tiles, the first of them in the list, shares of the rows
};
// What a row tile sees: smallest and largest position and first key.
struct __align__(16) WcRows {
  int pos_min, pos_max, lo_min, lo_max;
};
// What the sums know of a tile's rows.
struct __align__(16) WcFacts {
  float c[kWcRows];      // −tau·log2 e + log2 coef
  float near[kWcRows];   // c − slope·ahead
  float slope[kWcRows];  // −slope·log2 e
  float ahead[kWcRows];  // position less the tile's first row's
  int lo[kWcRows];       // first key of the row's document
  uint32_t counts[kWcRows / 32];  // rows that are there and add something
  int pos0, skip;        // position of the first row, and its head in the group
  int whole;             // all rows count
  float unit;            // what a value 1 of the packed queries stands for, a power of two
};
struct WcArgs {
  Q8WeighArgs a;
  WcSlot* slots;     // [n_seqs]
  long long* cum;    // [n_seqs + 1] segments before each slot
  WcRows* rows;      // [max_tiles]
  int* slot_of;      // [max_tiles]
  int* n_tiles;
  uint4* packed;     // [Hkv][max_tiles] tiles of 128 queries
  WcFacts* facts;    // [Hkv][max_tiles]
  int* done;         // [2·kWcTurns·blocks][8] shares of a warp's keys that are there
  float* part;       // [2·kWcTurns·blocks][256]
  int max_tiles, blocks;
};

struct WcSeg {
  WcSlot s;
  long long id, first;  // of the segment, and of its key tile's first share
  int kvh, kt, rt, rt_end;
  int key_min, key_max;  // of the tile's keys
  bool seen;             // some row may see some of them
  __device__ __forceinline__ int pages() const { return s.lnpre + s.npages - s.lwfirst; }
  __device__ __forceinline__ int page(int t) const { return t < s.lnpre ? t : t - s.lnpre + s.lwfirst; }
};
// The slots and their places, kept by a block where they are few.
constexpr int kWcFew = 32;
struct WcFew {
  WcSlot slots[kWcFew];
  long long cum[kWcFew + 1];
};
// Segment id; `slot` is the last one's slot (ids grow).
template <int P>
__device__ __forceinline__ WcSeg wc_seg(const WcArgs& g, const WcFew& sh, long long id, int& slot) {
  const bool few = g.a.b.n_seqs <= kWcFew;
  int lo = slot, hi = g.a.b.n_seqs - 1;
  if (few) {
    while (lo < hi && sh.cum[lo + 1] <= id) ++lo;
  } else {
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (__ldcg(g.cum + m) <= id) lo = m;
      else hi = m - 1;
    }
  }
  slot = lo;
  WcSeg x;
  const int4* p = reinterpret_cast<const int4*>(few ? sh.slots + lo : g.slots + lo);
#pragma unroll
  for (int i = 0; i < 4; ++i) reinterpret_cast<int4*>(&x.s)[i] = p[i];
  const long long cum = few ? sh.cum[lo] : __ldcg(g.cum + lo), off = id - cum, rest = div_line(off, x.s.T);
  x.kt = (int)(off - rest * x.s.T);
  const int sp = (int)div_line(rest, g.a.c.Hkv);
  x.kvh = (int)(rest - (long long)sp * g.a.c.Hkv);
  x.id = id;
  x.first = cum + (long long)x.kvh * x.s.T + x.kt;
  x.rt = (int)div_line((long long)x.s.nrt * sp, x.s.nsplit);
  x.rt_end = (int)div_line((long long)x.s.nrt * (sp + 1), x.s.nsplit);
  constexpr int PT = kWcKeys / P;
  const int p0 = x.page(x.kt * PT), p1 = x.page(min((x.kt + 1) * PT, x.pages()) - 1);
  x.key_min = p0 * P;
  x.key_max = min(p1 * P + P, x.s.L) - 1;
  x.seen = p0 < x.s.npre || p1 >= x.s.wfirst;
  return x;
}
// Of the 32 row tiles from rt on, those that may see the segment's keys, and those all of whose rows see them all.
struct WcMask {
  uint32_t some, all;
};
__device__ __forceinline__ void wc_sees(const WcArgs& g, const WcSeg& x, int rt, bool& some, bool& all) {
  some = all = false;
  if (rt < x.rt_end) {
    const int4 r = __ldcg(reinterpret_cast<const int4*>(g.rows + x.s.rt0 + rt));
    some = (r.y >= x.key_min && r.z <= x.key_max) || x.key_min < x.s.pre;
    all = r.x >= x.key_max && (r.w <= x.key_min || x.key_max < x.s.pre);
  }
}
__device__ __forceinline__ WcMask wc_mask(const WcArgs& g, const WcSeg& x, int rt) {
  bool some, all;
  wc_sees(g, x, rt + (threadIdx.x & 31), some, all);
  return WcMask{__ballot_sync(0xffffffffu, some), __ballot_sync(0xffffffffu, all)};
}

// A segment as the warps find it in shared memory: its pages, and the first 32 row tiles' bits.
struct __align__(16) WcPage {
  int at, key0;  // page · KV heads + KV head, first key; kNoKey: no page
  float ks;
  int pad;
};
struct __align__(16) WcInfo {
  WcSeg x;
  WcMask mask;
  WcPage pages[kWcKeys / 16];
};

// 16 columns of the thread's lane, and the tie of their values behind a wait.
__device__ __forceinline__ void tm_ask16(uint32_t addr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tm_tie16(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}

// D fp32, A and B halves, both along K; M = 128.
__device__ __forceinline__ uint32_t instr_desc_half(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
template <bool I8, int D, int P, bool capped, bool biased>
__global__ void __launch_bounds__(kWcThreads, 1) weigh_chunk_kernel(WcArgs g) {
  pdl_enter();
  constexpr int HALF = 128 * D * 2;      // bytes of 128 keys or rows
  constexpr int PT = kWcKeys / P;        // pages a key tile
  extern __shared__ __align__(128) unsigned char dyn_sm[];
  __shared__ uint64_t q_full[kWcQ], q_empty[kWcQ], f_full[kWcMeta], k_full[kWcK], k_empty[kWcK], s_full[2][2], s_empty[2][2];
  __shared__ uint64_t g_full[kWcSegs], g_empty[kWcSegs], x_full[2], x_empty[2];
  __shared__ uint32_t tm_base;
  __shared__ WcFacts facts[kWcMeta];
  __shared__ WcInfo segs[kWcSegs];
  __shared__ float x_sum[2][kWcKeys];  // the second rows' sums, of a segment and the next
  __shared__ volatile int gave_up;
  __shared__ WcFew few;
  const Q8WeighArgs& a = g.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
  const uint32_t sm0 = (smem_u32(dyn_sm) + 1023u) & ~1023u;
  const uint32_t k_sm = sm0, q_sm = sm0 + kWcK * 2 * HALF;
  if (tid == 0) {
    for (int i = 0; i < kWcQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 2);
    }
    for (int i = 0; i < kWcMeta; ++i) mbar_init(&f_full[i], 1);
    for (int i = 0; i < kWcSegs; ++i) {
      mbar_init(&g_full[i], 1);
      mbar_init(&g_empty[i], 27);  // 16 warps of sums, 8 of keys, 2 of products, 1 of rows
    }
    for (int i = 0; i < kWcK; ++i) {
      mbar_init(&k_full[i], 256);
      mbar_init(&k_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i][0], 2);  // the products, and the thread that issued them: it has waited for the rows' facts
      mbar_init(&s_full[i][1], 2);
      mbar_init(&s_empty[i][0], 256);
      mbar_init(&s_empty[i][1], 256);
      mbar_init(&x_full[i], 256);
      mbar_init(&x_empty[i], 256);
    }
    gave_up = 0;
    mbar_fence_init();
  }
  if (warp == 24) tm_alloc(&tm_base);
  if (a.b.n_seqs <= kWcFew) {
    for (int i = tid; i < a.b.n_seqs * 4; i += kWcThreads)
      reinterpret_cast<int4*>(few.slots)[i] = __ldcg(reinterpret_cast<const int4*>(g.slots) + i);
    if (tid <= a.b.n_seqs) few.cum[tid] = __ldcg(g.cum + tid);
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = tm_base;  // sums of stage s and half h at columns 256·s + 128·h
  const long long n_segs = g.cum[a.b.n_seqs];
  const int G = a.c.G, Hkv = a.c.Hkv;
  auto wait = [&](uint64_t* bar, int phase) -> bool {  // a wait that runs out of its bound stops every role
    if (mbar_wait_second(bar, (uint32_t)(phase & 1))) return true;
    gave_up = 1;
    return false;
  };
  auto wait_warp = [&](uint64_t* bar, int phase) -> bool { return __all_sync(0xffffffffu, wait(bar, phase)); };
  int slot = 0, u = 0;  // units (row tiles against key tiles) so far, the same for every role
  bool ok = true;
  // the k-th segment of the block, once it is there; given back with seg_done
  auto seg_wait = [&](int k) -> bool { return wait_warp(&g_full[k % kWcSegs], k / kWcSegs); };
  auto seg_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&g_empty[k % kWcSegs]);
  };
  auto seg_mask = [&](const WcInfo& q, int rt) { return rt == q.x.rt ? q.mask : wc_mask(g, q.x, rt); };
  const int n_mine = blockIdx.x < n_segs ? (int)((n_segs - 1 - blockIdx.x) / gridDim.x) + 1 : 0;

  // Registers after the splits below: 512 x 80 + 256 x 64 + 128 x 48 = 63488; launched with 896 x 72 = 64512.
  if (wg < 4) {  // ------------------------------------------------ sums: two threads a key
    asm volatile("setmaxnreg.inc.sync.aligned.u32 80;\n");
    const int half = wg & 1, part = wg >> 1;  // of the keys, and of a tile's rows
    const int ks_ = 128 * half + (tid & 127);
    const uint32_t s_tm = tm + ((uint32_t)(32 * (warp & 3)) << 16) + 128 * half;
    for (int k = 0; k < n_mine && ok; ++k) {
      if (!seg_wait(k)) {
        ok = false;
        break;
      }
      const WcInfo& q = segs[k % kWcSegs];
      const WcPage page = q.pages[ks_ / P];
      const int key = page.key0 + ks_ % P, pre = q.x.s.pre;
      const bool there = key < q.x.s.L;
      const float k1 = page.ks * a.sc.scale * (capped ? a.sc.inv_cap : kLog2e), out = a.sc.cap * kLog2e;
      float* wp = a.w + (size_t)page.at * P + ks_ % P;
      const bool reads = part == 0 && there && key < q.x.s.fresh && a.decay != 0.0f;
      float before = 0.0f;
      if (reads && q.x.s.nsplit == 1) before = *wp;
      unsigned long long acc[4] = {0ull, 0ull, 0ull, 0ull};
      for (int rt = q.x.rt; rt < q.x.rt_end && ok && q.x.seen; rt += 32) {
        WcMask m = seg_mask(q, rt);
        for (; m.some; m.some &= m.some - 1u, ++u) {
          const int i = __ffs(m.some) - 1, st = u & 1, ms = u % kWcMeta;
          const WcFacts& f = facts[ms];
          const int n_rows = min(kWcRows, q.x.s.count * G - (rt + i) * kWcRows);
          if (!wait_warp(&s_full[st][half], u >> 1)) {
            ok = false;
            break;
          }
          tm_fence_after();
          const bool whole = (m.all >> i & 1u) && f.whole;
          const unsigned long long k2 = f2_splat(k1 * f.unit);
          const float away = (float)(f.pos0 - key);  // (of the tile's first row; used where it is not negative)
          // 16 rows: their raw sums to weights, added up; `bits` are the rows that see the key
          auto weigh = [&](int c0, const float (&raw)[16], bool whole, uint32_t bits) {
            unsigned long long t2[8];
            if (capped) {  // y = raw·k, then cap·log2 e·y·T(y²)
              unsigned long long z2[8];
              float b4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
              for (int n = 0; n < 8; ++n) {
                t2[n] = f2_mul(f2_pack(raw[2 * n], raw[2 * n + 1]), k2);
                z2[n] = f2_mul(t2[n], t2[n]);
                float y0, y1;
                f2_unpack(z2[n], y0, y1);
                b4[n & 3] = max3(b4[n & 3], y0, y1);
              }
              const float big = max3(max3(b4[0], b4[1], b4[2]), b4[3], 0.0f);
              constexpr TanhPoly poly = tanh_poly();
              if (__all_sync(0xffffffffu, big <= 1.0f)) {
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                  unsigned long long r = f2_fma(z2[n], f2_splat(poly.far[6]), f2_splat(poly.far[5]));
#pragma unroll
                  for (int e = 4; e >= 0; --e) r = f2_fma(r, z2[n], f2_splat(poly.far[e]));
                  t2[n] = f2_mul(f2_mul(r, f2_splat(out)), t2[n]);
                }
              } else {
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                  float y0, y1;
                  f2_unpack(t2[n], y0, y1);
                  t2[n] = f2_mul(f2_pack(tanh_fine(y0), tanh_fine(y1)), f2_splat(out));
                }
              }
            }
            // in steps, so that no row's chain waits for another's
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const bool near = biased && whole;
              const float4 c = *reinterpret_cast<const float4*>((near ? f.near : f.c) + c0 + 4 * n);
              unsigned long long a0 = f2_pack(c.x, c.y), a1 = f2_pack(c.z, c.w);
              if (biased) {
                const float4 sl = *reinterpret_cast<const float4*>(f.slope + c0 + 4 * n);
                unsigned long long d0 = f2_splat(away), d1 = d0;
                if (!whole) {  // (a prefix' keys may lie behind the row)
                  const float4 ah = *reinterpret_cast<const float4*>(f.ahead + c0 + 4 * n);
                  d0 = f2_pack(fabsf(ah.x + away), fabsf(ah.y + away));
                  d1 = f2_pack(fabsf(ah.z + away), fabsf(ah.w + away));
                }
                a0 = f2_fma(f2_pack(sl.x, sl.y), d0, a0);
                a1 = f2_fma(f2_pack(sl.z, sl.w), d1, a1);
              }
              t2[2 * n] = capped ? f2_add(t2[2 * n], a0) : f2_fma(f2_pack(raw[4 * n], raw[4 * n + 1]), k2, a0);
              t2[2 * n + 1] = capped ? f2_add(t2[2 * n + 1], a1) : f2_fma(f2_pack(raw[4 * n + 2], raw[4 * n + 3]), k2, a1);
            }
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              float e0, e1;
              f2_unpack(t2[n], e0, e1);
              if (!whole) {
                if (!(bits >> (2 * n) & 1u)) e0 = -CUDART_INF_F;
                if (!(bits >> (2 * n + 1) & 1u)) e1 = -CUDART_INF_F;
              }
              t2[n] = f2_pack(ex2f(e0), ex2f(e1));
            }
#pragma unroll
            for (int n = 0; n < 8; ++n) acc[n & 3] = f2_add(acc[n & 3], t2[n]);
          };
          const uint32_t from = s_tm + 256 * st;
          const int c0 = 64 * part;
          if (whole) {  // (straight on, so that the sums stay where the loads put them)
            float raw[4][16];
            tm_ask16(from + c0, raw[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              tm_wait_ld();
              tm_tie16(raw[c]);
              if (c < 3) tm_ask16(from + c0 + 16 * (c + 1), raw[c + 1]);
              weigh(c0 + 16 * c, raw[c], true, 0xffffffffu);
            }
          } else {
            // Rows lie in the order of their positions: those from the key's own on see it, up to the window's end.
            int j0 = min(max(key - f.pos0, -1), kWcRows) * G - f.skip, j1 = kWcRows;
            if (a.sc.window > 0)
              j1 = (int)min(max((long long)key + a.sc.window - f.pos0, -1LL), (long long)kWcRows) * G - f.skip;
            if (key < pre) {
              j0 = 0;
              j1 = kWcRows;
            }
            auto below = [](int n) { return n <= 0 ? 0u : n >= 16 ? 0xffffu : (1u << n) - 1u; };
#pragma unroll 1
            for (int c = c0; c < min(n_rows, c0 + 64); c += 16) {
              uint32_t bits = f.counts[c / 32] >> (c & 16) & below(j1 - c) & ~below(j0 - c);
              if (a.sc.first_key && key >= pre) {
#pragma unroll 4
                for (int n = 0; n < 16; ++n)
                  if (f.lo[c + n] > key) bits &= ~(1u << n);
              }
              if (!__any_sync(0xffffffffu, bits != 0u)) continue;
              float raw[16];
              tm_ask16(from + c, raw);
              tm_wait_ld();
              tm_tie16(raw);
              weigh(c, raw, false, bits);
            }
          }
          tm_fence_before();
          mbar_arrive(&s_empty[st][half]);
        }
      }
      if (!ok) break;
      float sum = f2_sum(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])));
      const int b = k & 1;
      if (part) {
        if (k >= 2 && !wait_warp(&x_empty[b], (k >> 1) - 1)) {
          ok = false;
          break;
        }
        x_sum[b][ks_] = sum;
        mbar_arrive(&x_full[b]);
        seg_done(k);
        continue;
      }
      if (!wait_warp(&x_full[b], k >> 1)) {
        ok = false;
        break;
      }
      sum += x_sum[b][ks_];
      mbar_arrive(&x_empty[b]);
      const int nsplit = q.x.s.nsplit;
      const long long id = q.x.id, first = q.x.first, T = q.x.s.T;
      seg_done(k);
      if (nsplit > 1) {
        // each warp for its own keys: the one that comes last adds the shares, in their order
        g.part[id * kWcKeys + ks_] = sum;
        __threadfence();
        __syncwarp();
        int last = 0;
        if (lane == 0) last = atomicAdd(g.done + first * 8 + warp, 1) == nsplit - 1;
        if (!__shfl_sync(0xffffffffu, last, 0)) continue;
        __threadfence();
        sum = 0.0f;
        for (int i = 0; i < nsplit; ++i) sum += __ldcg(g.part + (first + (long long)i * Hkv * T) * kWcKeys + ks_);
        if (reads) before = *wp;
      }
      if (there) *wp = fmaf(before, a.decay, sum);
    }
  } else if (wg < 6) {  // ------------------------------------------------ keys
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    const int cw = warp - 16;                      // keys 32·cw .. 32·cw + 31 of a tile
    constexpr int CPR = D / 16;                   // 16-code chunks of a key
    constexpr int RPI = 32 / CPR, NI = 32 / RPI;  // keys a load, loads of a warp's keys
    // (as in the chunk attention: eight lanes store to eight banks' quads)
    const int cch = D == 128 ? (lane & 3) | (lane >> 1 & 4) : lane % CPR;
    const int crow = D == 128 ? (lane >> 2 & 1) | (lane >> 3 & 2) : lane / CPR;
    uint4 codes[NI];
    auto load = [&](const WcInfo& q) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int rr = i * RPI + crow, tk = rr % P;
        const WcPage page = q.pages[(32 * cw + rr) / P];
        codes[i] = make_uint4(0u, 0u, 0u, 0u);
        if (page.key0 + tk < q.x.s.L)  // (false where there is no page)
          codes[i] = __ldg(reinterpret_cast<const uint4*>(a.c.k_pool + ((size_t)page.at * P + tk) * D + cch * 16));
      }
    };
    int tiles = 0;  // key tiles so far
    for (int k = 0; k < n_mine && ok; ++k) {
      if (!seg_wait(k)) {
        ok = false;
        break;
      }
      const WcInfo& q = segs[k % kWcSegs];
      const bool seen = q.x.seen;
      if (seen) load(q);
      seg_done(k);
      if (!seen) continue;
      if (tiles >= kWcK && !wait_warp(&k_empty[tiles % kWcK], tiles / kWcK - 1)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int rr = 32 * (cw & 3) + i * RPI + crow;
        const uint32_t dst = k_sm + (tiles % kWcK * 2 + (cw >> 2)) * HALF;
        uint4 h0, h1;
        codes_half<I8, false>(codes[i].x, h0.x, h0.y);
        codes_half<I8, false>(codes[i].y, h0.z, h0.w);
        codes_half<I8, false>(codes[i].z, h1.x, h1.y);
        codes_half<I8, false>(codes[i].w, h1.z, h1.w);
        sts128(dst + tile_off(rr, 2 * cch), h0);
        sts128(dst + tile_off(rr, 2 * cch + 1), h1);
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      mbar_arrive(&k_full[tiles % kWcK]);
      ++tiles;
    }
  } else {  // ------------------------------------------------ products, and the rows' copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;\n");
    if (warp < 26) {  // a warp a half of the keys, one elected thread of it
      const int h = warp - 24;
      const uint64_t k_desc = smem_desc(k_sm + h * HALF, 16, 1024), q_desc = smem_desc(q_sm, 16, 1024);
      int tiles = 0;
      for (int k = 0; k < n_mine && ok; ++k) {
        if (!seg_wait(k)) {
          ok = false;
          break;
        }
        const WcInfo& q = segs[k % kWcSegs];
        if (q.x.seen) {
          ok = wait_warp(&k_full[tiles % kWcK], tiles / kWcK);
          const uint64_t k_tile = k_desc + (uint32_t)(tiles % kWcK * (2 * HALF >> 4));
          tm_fence_after();
          for (int rt = q.x.rt; rt < q.x.rt_end && ok; rt += 32) {
            WcMask m = seg_mask(q, rt);
            for (; m.some; m.some &= m.some - 1u, ++u) {
              const int i = __ffs(m.some) - 1, st = u & 1, qs = u % kWcQ;
              const int n_rows = min(kWcRows, q.x.s.count * G - (rt + i) * kWcRows);
              if (!wait_warp(&f_full[u % kWcMeta], u / kWcMeta) || !wait_warp(&q_full[qs], u / kWcQ) ||
                  (u >= 2 && !wait_warp(&s_empty[st][h], (u >> 1) - 1))) {
                ok = false;
                break;
              }
              tm_fence_after();
              if (elect_one()) {
                const uint32_t id_s = instr_desc_half((n_rows + 15) / 16 * 16);
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {  // (addresses advance in units of 16 bytes)
                  const uint32_t o = ((n >> 2) * 16384 + (n & 3) * 32) >> 4;
                  mma_ss(tm + 256 * st + 128 * h, k_tile + o, q_desc + (uint32_t)(qs * (HALF >> 4)) + o, id_s, n > 0);
                }
                tm_commit(&s_full[st][h]);
                mbar_arrive(&s_full[st][h]);
                tm_commit(&q_empty[qs]);
              }
              __syncwarp();
            }
          }
          if (ok && elect_one()) tm_commit(&k_empty[tiles % kWcK]);
          __syncwarp();
          ++tiles;
        }
        seg_done(k);
      }
    } else if (warp == 26) {
      for (int k = 0; k < n_mine && ok; ++k) {
        if (!seg_wait(k)) {
          ok = false;
          break;
        }
        const WcInfo& q = segs[k % kWcSegs];
        for (int rt = q.x.rt; rt < q.x.rt_end && ok && q.x.seen; rt += 32) {
          WcMask m = seg_mask(q, rt);
          for (; m.some; m.some &= m.some - 1u, ++u) {
            const int i = __ffs(m.some) - 1, st = u % kWcQ, ms = u % kWcMeta;
            if (u >= kWcQ && !wait_warp(&q_empty[st], u / kWcQ - 1)) {
              ok = false;
              break;
            }
            if (elect_one()) {
              const size_t at = (size_t)q.x.kvh * g.max_tiles + q.x.s.rt0 + rt + i;
              mbar_expect_tx(&q_full[st], HALF);
              bulk_g2s(dyn_sm + (q_sm - smem_u32(dyn_sm)) + st * HALF, g.packed + at * (HALF / 16), HALF, &q_full[st]);
              mbar_expect_tx(&f_full[ms], sizeof(WcFacts));
              bulk_g2s(&facts[ms], g.facts + at, sizeof(WcFacts), &f_full[ms]);
            }
            __syncwarp();
          }
        }
        if (ok) seg_done(k);
      }
      // what was asked for lands before the block ends, whatever gave up
      if (!ok || gave_up) {
        for (int k = max(0, u - kWcQ); k < u; ++k) mbar_wait_second(&q_full[k % kWcQ], (uint32_t)(k / kWcQ & 1));
        for (int k = max(0, u - kWcMeta); k < u; ++k) mbar_wait_second(&f_full[k % kWcMeta], (uint32_t)(k / kWcMeta & 1));
      }
    } else {
      // Segments, as far ahead as there is room, two at a time: a look-up is a chain of divisions and loads, longer than
      // the work with a segment of few row tiles. A half of the warp has one each.
      const int side = lane >> 4, l16 = lane & 15;
      auto halves = [&](bool b0, bool b1) {  // a half's 16 bits of each
        const uint32_t v0 = __ballot_sync(0xffffffffu, b0), v1 = __ballot_sync(0xffffffffu, b1);
        return (v0 >> (16 * side) & 0xffffu) | (v1 >> (16 * side)) << 16;
      };
      for (int k = 0; k < n_mine && ok; k += 2) {
        const WcSeg x = wc_seg<P>(g, few, blockIdx.x + (long long)min(k + side, n_mine - 1) * gridDim.x, slot);
        WcPage page{0, kNoKey, 0.0f, 0};
        const int t = x.kt * PT + l16;
        if (l16 < PT && t < x.pages()) {
          const int ph = phys_page(a.c.block_table, x.s.seq, x.page(t), a.c.maxp, a.c.nphys, a.c.status);
          if (ph >= 0) {
            page.at = ph * Hkv + x.kvh;
            page.key0 = x.page(t) * P;
            page.ks = a.c.k_scale[page.at];
          }
        }
        bool some[2], all[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) wc_sees(g, x, x.rt + 16 * i + l16, some[i], all[i]);
        const WcMask mask{halves(some[0], some[1]), halves(all[0], all[1])};
        for (int j = 0; j < 2 && k + j < n_mine; ++j) {
          if (k + j >= kWcSegs && !wait_warp(&g_empty[(k + j) % kWcSegs], (k + j) / kWcSegs - 1)) {
            ok = false;
            break;
          }
          WcInfo& q = segs[(k + j) % kWcSegs];
          if (side == j) {
            if (l16 < PT) q.pages[l16] = page;
            if (l16 == 0) {
              q.x = x;
              q.mask = mask;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&g_full[(k + j) % kWcSegs]);
        }
      }
    }
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  if (warp == 24) tm_free(tm);
  if (tid == 0 && gave_up) raise_flag(a.c.status, ENTMAXKV_DEV_TIMEOUT);
}

// The product kernel for one code type and head dimension (a translation unit each).
template <bool I8, int D>
cudaError_t weigh_chunk_run(const WcArgs& g, cudaStream_t st);

template <bool I8, int D, int P, bool CAP, bool BIAS>
cudaError_t weigh_chunk_start(const WcArgs& g, cudaStream_t st) {
  const int smem = (2 * kWcK + kWcQ) * 128 * D * 2 + 1024;
  const cudaError_t e = ensure_smem((const void*)weigh_chunk_kernel<I8, D, P, CAP, BIAS>, smem);
  if (e != cudaSuccess) return e;
  return launch_k(true, weigh_chunk_kernel<I8, D, P, CAP, BIAS>, dim3(g.blocks), dim3(kWcThreads), (size_t)smem, st, g);
}
template <bool I8, int D, int P>
cudaError_t weigh_chunk_form(const WcArgs& g, cudaStream_t st) {
  const bool cap = g.a.sc.cap > 0.0f, bias = g.a.sc.slopes != nullptr;
  if (cap) return bias ? weigh_chunk_start<I8, D, P, true, true>(g, st) : weigh_chunk_start<I8, D, P, true, false>(g, st);
  return bias ? weigh_chunk_start<I8, D, P, false, true>(g, st) : weigh_chunk_start<I8, D, P, false, false>(g, st);
}
template <bool I8, int D>
cudaError_t weigh_chunk_pages(const WcArgs& g, cudaStream_t st) {
  return g.a.c.P == 32 ? weigh_chunk_form<I8, D, 32>(g, st) : weigh_chunk_form<I8, D, 16>(g, st);
}

}  // namespace ekv
