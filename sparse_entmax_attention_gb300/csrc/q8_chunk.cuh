// q8_chunk.cuh -- softmax attention of many new tokens a sequence over the 8-bit
// paged cache (prompt chunks, mixed batches) on the fifth-generation tensor
// cores.
//
// An item is 256 rows of one (slot, KV head): rows are (token, head of the
// group), so a K/V tile serves the whole group. Per tile of 128 keys (the
// pages of the item's span in order):
//   S = Q·K^T          128 rows × 64 keys a product, Q and the codes as halves
//                      (both exact: a power of two per query row), fp32 sums in
//                      tensor memory;
//   t = S·ks·scale·log2 e (capped, biased, masked) + log2 vs, one row a thread;
//   w = 2^{t − M + 8}  as halves (off by 2^-11, an eighth of the bf16 output's
//                      rounding) into tensor memory over S, M a running bound of
//                      the row's maximum that is moved when the maximum passes it
//                      by 6: w ≤ 2^14, and weights down to 2^-32 of the largest
//                      survive the rounding;
//   O += w·codes       accumulated in tensor memory, rescaled when M moves.
// The V scale rides in w, so Σp is Σ over pages of (Σ w)/vs, of unrounded w.
//
// Warps: 4 + 4 softmax (a thread a row), 4 converters (codes from L2 through
// registers into swizzled half tiles, two stages), 2 that issue the products, one
// for each 128 rows. A row's softmax takes 64 keys at a time, the last ones first,
// so that while it is at one half of a tile's keys the other half's products run.
// All items form one line (KV head outermost) cut into equal pieces for
// one block a multiprocessor; an item cut in two leaves (M, Σp, O) pieces that a
// second kernel joins in the order of the line.
//
// Bound: the latency of the softmax warps, two a scheduler. Of a tile's 2600 cycles of products
// (measured alone; 2050 in turns of 128 keys) the capped form takes about 5400:
// fp32 pipe 44% busy, tensor pipe 37%, IPC 2.3, the rest the latency of each
// row's chain (maxima in one chain instead of four: 8% slower). Measured, int8, 8
// KV heads of 4 query heads, d = 128: 2048 tokens behind 30001, capped (1.04
// TFLOP), 1.18 ms, 885 TFLOP/s; behind 8000 without a cap 289 us. One
// thread that issued all products, and tiles in turns of 128 keys, took 1.54 ms:
// issuing one costs a thread about 75 cycles, more than the product.
#pragma once

#include "q8_tiles.cuh"

namespace ekv {

constexpr int kChunkThreads = 512;
constexpr int kChunkRows = 256;
constexpr int kChunkKeys = 128;
constexpr int kChunkMaxBlocks = 256;
// What an item costs beside its tiles, in tiles: its place, queries and answers
// (14 to 16 thousand cycles against 4500 to 5400 a tile). Items have that many
// places on the line in front of their tiles', so that blocks of many short items
// get fewer tiles (six prompts' chunks of 97-token documents, e4m3, slopes: 134 us
// without them, 109 with).
constexpr int kChunkItem = 3;

// What the roles know of an item, filled in once by the listing kernel.
struct __align__(16) ChunkItem {
  int slot, rt, T, Tp;                // its tiles and pages
  int seq, L, start, count;           // Q8Slot
  int pre, npre, wfirst, npages;      // Q8Span
};
struct ChunkArgs {
  Q8AttendArgs a;
  ChunkItem* items;
  int* cum;        // [n_items + 1] places of one KV head's line before each item
  int* n_items;    // [2] items, and those of them without a tile
  int* empty;      // the latter
  int2* cuts;      // [blocks] (item, KV head) that a block begins inside of; item −1: at one's start
  float* part_o;   // [blocks][2][256][D]
  float2* part_ml; // [blocks][2][256]
  int max_items, blocks;
};

// The span of item (slot, rt): its tokens' pages.
__device__ __forceinline__ Q8Span chunk_span(const Q8AttendArgs& a, const Q8Slot& s, int b, int rt) {
  const int t0 = rt * kChunkRows / a.c.G, t1 = min(s.count, (rt * kChunkRows + kChunkRows - 1) / a.c.G + 1);
  return q8_span(a.c, a.sc, s, b, t0, t1 - t0);
}

// ---------------------------------------------------------------------------
// tensor memory and products

__device__ __forceinline__ void tm_alloc(uint32_t* out) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(out)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tm_free(uint32_t base) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(base) : "memory");
}
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tm_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// 32 columns of the thread's lane.
__device__ __forceinline__ void tm_ld32(uint32_t addr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// The values of earlier loads are read behind the wait that this follows.
__device__ __forceinline__ void tm_tie32(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
// 16 columns, read behind their own wait, and written.
__device__ __forceinline__ void tm_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n" ::"r"(
          r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

// Shared-memory descriptors of a half tile with 128-byte swizzle. Rows of 64
// halves (128 bytes) lie in groups of 8 (1024 bytes); a 128-wide tile is two
// such halves, `half` bytes apart. Bits: address/16, leading and stride byte
// offsets/16, version 1, swizzle 2 (128 bytes).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// D fp32, A and B halves; M = 128; B rows along K (mn = 0) or along N (mn = 1).
__device__ __forceinline__ constexpr uint32_t instr_desc(int n, int mn) {
  return (1u << 4) | ((uint32_t)mn << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

// Byte offset of 16-byte chunk ch (8 halves) of row t in a tile of 128 rows.
__device__ __forceinline__ uint32_t tile_off(int t, int ch) {
  return (uint32_t)((ch >> 3) * 16384 + t * 128 + (((ch & 7) ^ (t & 7)) << 4));
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A block's part of one item: `n` tiles, tile t0 + n − 1 first, `skip` places on.
// (Nearest keys come first, so that with a distance bias the first maximum is the
// last one.) n = 0: the block's line ends before the item's tiles.
struct ChunkSeg {
  int kvh, item, slot, rt, t0, n, T, skip;
  Q8Slot s;
  Q8Span sp;
};
// The part that begins at w; `item` is looked for from the start of the list
// (item < 0) or is the one behind the part before.
__device__ __forceinline__ ChunkSeg chunk_seg(const ChunkArgs& g, long long w, long long w_end, int S, int n_items,
                                              int item) {
  ChunkSeg x;
  x.kvh = (int)(w / S);
  const int off = (int)(w - (long long)x.kvh * S);
  if (item < 0) {
    int lo = 0, hi = n_items - 1;  // the last item that begins at or before `off`
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (g.cum[m] <= off) lo = m;
      else hi = m - 1;
    }
    item = lo;
  } else if (item == n_items) {
    item = 0;
  }
  ChunkItem it;
  for (;; item = item + 1 < n_items ? item + 1 : 0) {  // (items without a tile are passed over; some item has one)
    const int4* p = reinterpret_cast<const int4*>(g.items + item);
    *reinterpret_cast<int4*>(&it) = __ldcg(p);
    *(reinterpret_cast<int4*>(&it) + 1) = __ldcg(p + 1);
    *(reinterpret_cast<int4*>(&it) + 2) = __ldcg(p + 2);
    if (it.T > 0) break;
  }
  x.item = item;
  x.slot = it.slot;
  x.rt = it.rt;
  const int at = off - __ldcg(g.cum + item) - kChunkItem;
  x.t0 = max(at, 0);
  x.skip = max(-at, 0);
  x.T = it.T;
  x.n = (int)max(0LL, min((long long)(x.T - x.t0), w_end - w - x.skip));
  x.s = Q8Slot{it.seq, it.L, it.start, it.count};
  x.sp = Q8Span{it.pre, it.npre, it.wfirst, it.npages, it.Tp};
  return x;
}

struct PageMeta {
  float ks, lv, ivs;  // K scale, log2 of the V scale, its inverse
  int key0;           // first key; beyond every key where there is no page
};

template <bool I8, int D, int P, bool capped, bool biased, bool paired>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_kernel(ChunkArgs g) {
  pdl_enter();
  constexpr int KP = kChunkKeys / P;           // pages a tile
  constexpr int TILE = kChunkKeys * D * 2;     // bytes of a half tile
  extern __shared__ __align__(128) unsigned char dyn_sm[];
  __shared__ uint64_t q_full, o_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2][2], p_full[2][2];
  __shared__ uint32_t tm_base;
  __shared__ PageMeta meta[4][KP];
  __shared__ volatile int gave_up;
  const Q8AttendArgs& a = g.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
  const uint32_t sm0 = (smem_u32(dyn_sm) + 1023u) & ~1023u;
  const uint32_t q_sm = sm0, k_sm = sm0 + 2 * TILE, v_sm = sm0 + 4 * TILE;
  if (tid == 0) {
    mbar_init(&q_full, 256);
    mbar_init(&o_full, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 128);
      mbar_init(&v_full[i], 128);
      mbar_init(&k_empty[i], 2);
      mbar_init(&v_empty[i], 2);
      for (int c = 0; c < 2; ++c) {
        mbar_init(&s_full[i][c], 1 + c);  // (scored)
        mbar_init(&p_full[i][c], 128);
      }
    }
    gave_up = 0;
    mbar_fence_init();
  }
  if (warp == 12) tm_alloc(&tm_base);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = tm_base;  // S of the two halves at columns 0 and 128, O at 256 and 256 + D
  const int n_items = *g.n_items;
  const int S = n_items ? g.cum[n_items] : 0;
  const long long W = (long long)S * a.c.Hkv, nb = max(1LL, min(W, (long long)gridDim.x));
  const long long w_begin = blockIdx.x < nb ? W * blockIdx.x / nb : 0;
  const long long w_end = blockIdx.x < nb ? W * (blockIdx.x + 1) / nb : 0;
  const int G = a.c.G, Hkv = a.c.Hkv;
  // a wait that runs out of its bound stops every role
  auto wait = [&](uint64_t* bar, int phase) -> bool {
    if (mbar_wait_second(bar, (uint32_t)(phase & 1))) return true;
    gave_up = 1;
    return false;
  };
  auto wait_warp = [&](uint64_t* bar, int phase) -> bool { return __all_sync(0xffffffffu, wait(bar, phase)); };

  // Registers after the splits below: 256 x 168 + 128 x 104 + 128 x 72 = 512 x 128, what the block was launched with.
  if (wg < 2) {  // ------------------------------------------------ softmax: a thread a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;\n");
    const int row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_tm = tm + lanes + 128 * wg, o_tm = tm + lanes + 256 + D * wg;
    int it = 0, seg = 0, tile = 0;  // phases of this half's sums, items and all tiles so far
    bool ok = true;
    int item = -1;
    for (long long w = w_begin; w < w_end && ok; ++seg) {
      const ChunkSeg x = chunk_seg(g, w, w_end, S, n_items, item);
      if (x.n == 0) break;
      item = x.item + 1;
      const int rho = x.rt * kChunkRows + 128 * wg + row, rows = x.s.count * G;
      const bool mine = rho < rows, half = x.rt * kChunkRows + 128 * wg < rows;
      const int tok = mine ? rho / G : 0, head = x.kvh * G + (mine ? rho % G : 0);
      float kc = 0.0f, slope = 0.0f;  // the raw sums' factor (times the page's K scale): log2 units, or of the cap
      int pos = -1, lo = 0;
      const long long q_at = (long long)(x.s.start + tok) * a.q.ts + (long long)head * a.q.hs;
      const long long o_at = (long long)(x.s.start + tok) * a.out.ts + (long long)(paired ? head >> 1 : head) * a.out.hs;
      const uint32_t rows_sm = q_sm + wg * TILE;  // this half's query tile, and its answers on their way out
      if (mine) {  // (asked for before the queries)
        pos = x.s.L - x.s.count + tok;
        if (a.sc.window > 0) lo = max(0, pos - a.sc.window + 1);
        if (a.sc.first_key) lo = max(lo, a.sc.first_key[x.s.start + tok]);
        if (biased) slope = a.sc.slopes[head] * kLog2e;
      }
      if (half) {
        // the warp's query rows as halves, CPR lanes a row, each row brought near 2^13 by a power of two
        constexpr int CPR = D / 8, RPI = 32 / CPR;
        const int ch = lane % CPR, sub = lane / CPR;
#pragma unroll
        for (int i0 = 0; i0 < CPR; i0 += 8) {
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rl = (i0 + i) * RPI + sub;
            const long long at = __shfl_sync(0xffffffffu, q_at, rl);
            const bool there = __shfl_sync(0xffffffffu, (int)mine, rl);
            v[i] = there ? *reinterpret_cast<const uint4*>(a.q.p + at + ch * 8) : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rl = (i0 + i) * RPI + sub;
            uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t m = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) m = __vmaxu2(m, u[j] & 0x7fff7fffu);
            m = max(m & 0xffffu, m >> 16);
#pragma unroll
            for (int o = 1; o < CPR; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            int e = (int)(m >> 7) - 127;
            e = max(e, -100);
            // (a row with an infinity or NaN is all NaN, as in q_half_frag)
            const float f = m >= 0x7f80u ? CUDART_NAN_F : __uint_as_float((uint32_t)(13 - e + 127) << 23);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __half2 h = __floats2half2_rn(bf_lo(u[j]) * f, bf_hi(u[j]) * f);
              u[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            sts128(rows_sm + tile_off(32 * (warp & 3) + rl, ch), make_uint4(u[0], u[1], u[2], u[3]));
            const int back = __shfl_sync(0xffffffffu, e, (lane % RPI) * CPR);  // rows 8·RPI of the warp in turn
            if (lane / RPI == i0 + i)
              kc = __uint_as_float((uint32_t)(back - 13 + 127) << 23) * a.sc.scale * (capped ? a.sc.inv_cap : kLog2e);
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      mbar_arrive(&q_full);
      const int pos_min = __reduce_min_sync(0xffffffffu, mine ? pos : 0x7fffffff);
      const int lo_max = __reduce_max_sync(0xffffffffu, lo);
      float M = -CUDART_INF_F, l = 0.0f;
      if (half) {
        for (int j = 0; j < x.n && ok; ++j) {
          const PageMeta* pg = meta[(tile + j) & 3];
          // 64 columns (keys 64c ..) from their raw sums to halves over the first of them
          auto weigh = [&](int c, const float (&raw)[64]) {
            unsigned long long t2[32];
            // exponents against the bound so far, so that they need no other pass
            const float base = M > -CUDART_INF_F ? kLift - M : 0.0f;
            float m4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int q = 0; q < 64 / P; ++q) {
              const PageMeta pm = pg[c * (64 / P) + q];
              unsigned long long* u = t2 + q * (P / 2);
              const float* v = raw + q * P;
              const bool past = pm.key0 + P - 1 <= pos_min;
              float add = pm.lv + base;
              if (biased && past) add = fmaf(-slope, (float)(pos - pm.key0), add);
              const unsigned long long k2 = f2_splat(pm.ks * kc), a2 = f2_splat(add);
              if (capped) {  // y = raw·k, then cap·log2 e·y·T(y²)
                unsigned long long z2[P / 2];
                float b4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < P / 2; ++i) {
                  u[i] = f2_mul(f2_pack(v[2 * i], v[2 * i + 1]), k2);
                  z2[i] = f2_mul(u[i], u[i]);
                  float y0, y1;
                  f2_unpack(z2[i], y0, y1);
                  b4[i & 3] = max3(b4[i & 3], y0, y1);
                }
                const float big = max3(max3(b4[0], b4[1], b4[2]), b4[3], 0.0f);
                constexpr TanhPoly poly = tanh_poly();
                const float out = a.sc.cap * kLog2e;
                if (__all_sync(0xffffffffu, big <= 0.25f)) {
                  const unsigned long long c0 = f2_splat(poly.near[0] * out), c1 = f2_splat(poly.near[1] * out),
                                           c2 = f2_splat(poly.near[2] * out), c3 = f2_splat(poly.near[3] * out);
#pragma unroll
                  for (int i = 0; i < P / 2; ++i)
                    u[i] = f2_fma(f2_fma(f2_fma(f2_fma(c3, z2[i], c2), z2[i], c1), z2[i], c0), u[i], a2);
                } else if (__all_sync(0xffffffffu, big <= 1.0f)) {
#pragma unroll
                  for (int i = 0; i < P / 2; ++i) {
                    unsigned long long r = f2_fma(z2[i], f2_splat(poly.far[6]), f2_splat(poly.far[5]));
#pragma unroll
                    for (int n = 4; n >= 0; --n) r = f2_fma(r, z2[i], f2_splat(poly.far[n]));
                    u[i] = f2_fma(f2_mul(r, f2_splat(out)), u[i], a2);
                  }
                } else {
#pragma unroll
                  for (int i = 0; i < P / 2; ++i) {
                    float y0, y1;
                    f2_unpack(u[i], y0, y1);
                    u[i] = f2_fma(f2_pack(soft_cap(y0, 1.0f, 1.0f), soft_cap(y1, 1.0f, 1.0f)), f2_splat(out), a2);
                  }
                }
              } else {
#pragma unroll
                for (int i = 0; i < P / 2; ++i) u[i] = f2_fma(f2_pack(v[2 * i], v[2 * i + 1]), k2, a2);
              }
              if (biased) {
                const unsigned long long two = f2_splat(2.0f), sl = f2_splat(slope);
                if (past) {
                  unsigned long long at = f2_pack(0.0f, 1.0f);
#pragma unroll
                  for (int i = 0; i < P / 2; ++i) {
                    u[i] = f2_fma(at, sl, u[i]);
                    at = f2_add(at, two);
                  }
                } else {
                  float y = (float)(pos - pm.key0);
#pragma unroll
                  for (int i = 0; i < P / 2; ++i) {
                    u[i] = f2_fma(f2_pack(-fabsf(y), -fabsf(y - 1.0f)), sl, u[i]);
                    y -= 2.0f;
                  }
                }
              }
              if (!((past && pm.key0 >= lo_max) || pm.key0 + P <= x.sp.pre)) {
                // one bit a key: those from lo to pos, and the prefix
                const int from = min(max(lo - pm.key0, 0), P), to = min(max(pos - pm.key0 + 1, 0), P);
                const int pre = min(max(x.sp.pre - pm.key0, 0), P);
                auto below = [](int n) { return n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
                const uint32_t bits = (below(to) & ~below(from)) | below(pre);
#pragma unroll
                for (int i = 0; i < P / 2; ++i) {
                  float y0, y1;
                  f2_unpack(u[i], y0, y1);
                  if (!(bits >> (2 * i) & 1u)) y0 = -CUDART_INF_F;
                  if (!(bits >> (2 * i + 1) & 1u)) y1 = -CUDART_INF_F;
                  u[i] = f2_pack(y0, y1);
                }
              }
#pragma unroll
              for (int i = 0; i < P / 2; ++i) {
                float y0, y1;
                f2_unpack(u[i], y0, y1);
                m4[i & 3] = max3(m4[i & 3], y0, y1);
              }
            }
            const float mx = max3(max3(m4[0], m4[1], m4[2]), m4[3], -CUDART_INF_F);
            // the bound moves when the maximum passes it by more than the slack: in an item's first columns, and
            // seldom behind them
            const bool move = M > -CUDART_INF_F ? mx > kLift + kSlack : mx > M;
            if (__any_sync(0xffffffffu, move)) {
              float f = 1.0f;
              if (move) {
                const float to = mx - base, less = kLift - mx;  // the new bound, and what it takes off
                f = ex2f(M - to);                               // 0 from -inf
                M = to;
#pragma unroll
                for (int i = 0; i < 32; ++i) t2[i] = f2_add(t2[i], f2_splat(less));
              }
              l *= f;
              if (j > 0 || c == 0) {
                // behind the product of the 64 keys before: the next commit to the other columns' barrier
                ok = wait_warp(&s_full[wg][c ^ 1], it + j + (c ^ 1));
                tm_fence_after();
#pragma unroll 1
                for (int i = 0; i < D / 16; ++i) {
                  uint32_t o[16];
                  tm_ld16(o_tm + 16 * i, o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                  tm_st16(o_tm + 16 * i, o);
                }
              }
            }
            uint32_t w32[32];
#pragma unroll
            for (int q = 0; q < 64 / P; ++q) {
              unsigned long long s2[2] = {0ull, 0ull};
#pragma unroll
              for (int i = 0; i < P / 2; ++i) {
                float e0, e1;
                f2_unpack(t2[q * (P / 2) + i], e0, e1);
                e0 = ex2f(e0);
                e1 = ex2f(e1);
                s2[i & 1] = f2_add(s2[i & 1], f2_pack(e0, e1));
                const __half2 h = __floats2half2_rn(e0, e1);
                w32[q * (P / 2) + i] = *reinterpret_cast<const uint32_t*>(&h);
              }
              l = fmaf(f2_sum(f2_add(s2[0], s2[1])), pg[c * (64 / P) + q].ivs, l);
            }
            tm_st32(s_tm + 64 * c, w32);
          };
#pragma unroll 1
          for (int c = 1; c >= 0; --c) {
            if (!ok || !wait_warp(&s_full[wg][c], it + j)) {
              ok = false;
              break;
            }
            tm_fence_after();
            float raw[64];
            tm_ld32(s_tm + 64 * c, raw);
            tm_ld32(s_tm + 64 * c + 32, raw + 32);
            tm_wait_ld();
            tm_tie32(raw);
            tm_tie32(raw + 32);
            weigh(c, raw);
            tm_wait_st();
            tm_fence_before();
            mbar_arrive(&p_full[wg][c]);
          }
        }
        // (the commits behind the last products, so that no phase is passed over)
        ok = ok && wait_warp(&s_full[wg][1], it + x.n) && wait_warp(&s_full[wg][0], it + x.n);
        it += x.n + 1;
      }
      if (!ok || !wait_warp(&o_full, seg)) {
        ok = false;
        break;
      }
      tm_fence_after();
      const bool whole = x.n == x.T;
      const int piece = 2 * blockIdx.x + (seg ? 1 : 0);
      const float inv = whole ? att_inv(l) : 1.0f;
      // a pair's rows lie in neighbouring lanes: both form y = first + second, and each stores half of the chunks to
      // the first one's row
      const bool pairs = paired && whole;
      float first = 0.0f, fn = 1.0f;
      if (pairs) {
        const float lam = mine ? a.lam[(long long)(x.s.start + tok) * a.lam_ts + (head >> 1)] : 0.0f;
        first = lane & 1 ? -lam * inv : inv;
        if (half && a.gain) {
          float down = 1.0f, sum2;
#pragma unroll 1
          for (bool again = false;; again = true) {  // (once more where a row's squares pass fp32)
            sum2 = 0.0f;
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              float o[32];
              tm_ld32(o_tm + 32 * i, o);
              tm_wait_ld();
              tm_tie32(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const float m = __fmul_rn(o[k], first), y = __fadd_rn(m, __shfl_xor_sync(0xffffffffu, m, 1)) * down;
                sum2 = fmaf(y, y, sum2);
              }
            }
            if (again || !__any_sync(0xffffffffu, diff_past(sum2))) break;
            if (diff_past(sum2)) down = kDiffDown;
          }
          fn = diff_norm(a, sum2, down);
        }
      }
      if (half) {
        // rows leave through the query tile, so that a warp writes whole rows: bf16 rows at once, fp32 pieces in
        // column blocks of 256 bytes too
        constexpr int LPR = D == 128 ? 16 : 8;  // lanes a bf16 row
        const int wrow = 32 * (warp & 3);
        float* pp = g.part_o + ((size_t)piece * kChunkRows + 128 * wg + wrow) * D;
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          float o[32];
          __syncwarp();
          tm_ld32(o_tm + 32 * i, o);
          tm_wait_ld();
          tm_tie32(o);
          if (pairs) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float m = __fmul_rn(o[k], first);
              o[k] = __fadd_rn(m, __shfl_xor_sync(0xffffffffu, m, 1));
              if (a.gain) o[k] *= fn * a.gain[32 * i + k];
            }
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              if ((k / 8 & 1) == (lane & 1))
                sts128(rows_sm + tile_off(row & ~1, 4 * i + k / 8),
                       make_uint4(bf2_rn(o[k], o[k + 1]), bf2_rn(o[k + 2], o[k + 3]), bf2_rn(o[k + 4], o[k + 5]),
                                  bf2_rn(o[k + 6], o[k + 7])));
          } else if (whole) {
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              sts128(rows_sm + tile_off(row, 4 * i + k / 8),
                     make_uint4(bf2_rn(o[k] * inv, o[k + 1] * inv), bf2_rn(o[k + 2] * inv, o[k + 3] * inv),
                                bf2_rn(o[k + 4] * inv, o[k + 5] * inv), bf2_rn(o[k + 6] * inv, o[k + 7] * inv)));
          } else {  // 32 columns are 128 bytes a row: 8 lanes a row
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              sts128(rows_sm + tile_off(row, k / 4), make_uint4(__float_as_uint(o[k]), __float_as_uint(o[k + 1]),
                                                                __float_as_uint(o[k + 2]), __float_as_uint(o[k + 3])));
            __syncwarp();
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const int rl = 4 * n + lane / 8;
              if (__shfl_sync(0xffffffffu, (int)mine, rl))
                *reinterpret_cast<uint4*>(pp + rl * D + 32 * i + 4 * (lane % 8)) =
                    lds128(rows_sm + tile_off(wrow + rl, lane % 8));
            }
          }
        }
        if (whole) {
          __syncwarp();
#pragma unroll 4
          for (int n = 0; n < LPR; ++n) {
            const int rl = n * (32 / LPR) + lane / LPR;
            const long long at = __shfl_sync(0xffffffffu, o_at, rl);
            if (__shfl_sync(0xffffffffu, (int)mine, rl) && !(pairs && (rl & 1)))
              *reinterpret_cast<uint4*>(a.out.p + at + 8 * (lane % LPR)) = lds128(rows_sm + tile_off(wrow + rl, lane % LPR));
          }
        }
        __syncwarp();
        if (mine) {
          if (!whole) g.part_ml[(size_t)piece * kChunkRows + 128 * wg + row] = make_float2(M - kLift, l);
          else if (a.tau) a.tau[(size_t)(x.s.start + tok) * Hkv * G + head] = att_lse(M - kLift, l);
        }
      }
      tm_fence_before();
      tile += x.n;
      w += x.skip + x.n;
    }
  } else if (wg == 2) {  // ------------------------------------------ converters
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;\n");
    const int cw = warp - 8;                      // rows 32·cw .. 32·cw + 31 of a tile
    constexpr int CPR = D / 16;                   // 16-code chunks of a row
    constexpr int RPI = 32 / CPR, NI = 32 / RPI;  // rows a load, loads of a warp's rows
    constexpr int PW = 32 / P;                    // pages of a warp's rows: 1 or 2
    // eight lanes store to eight banks' quads: at D = 128 four chunks of two rows, not eight of one, whose two 64-wide
    // halves would meet in the same banks
    const int cch = D == 128 ? (lane & 3) | (lane >> 1 & 4) : lane % CPR;
    const int crow = D == 128 ? (lane >> 2 & 1) | (lane >> 3 & 2) : lane / CPR;
    int it = 0;
    bool ok = true;
    int item = -1;
    for (long long w = w_begin; w < w_end && ok;) {
      const ChunkSeg x = chunk_seg(g, w, w_end, S, n_items, item);
      if (x.n == 0) break;
      item = x.item + 1;
      // 32 tiles' pages at once, a tile a lane
      int ph[PW], key[PW];
      float ks[PW], vs[PW];
      auto load = [&](const uint8_t* pool, int j, uint4 (&codes)[NI]) {
        int f[PW], k0[PW];
#pragma unroll
        for (int q = 0; q < PW; ++q) {
          f[q] = __shfl_sync(0xffffffffu, ph[q], j & 31);
          k0[q] = __shfl_sync(0xffffffffu, key[q], j & 31);
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int rr = i * RPI + crow, tk = rr % P;
          const int fq = rr < P ? f[0] : f[PW - 1], kq = rr < P ? k0[0] : k0[PW - 1];
          codes[i] = make_uint4(0u, 0u, 0u, 0u);
          if (kq + tk < x.s.L)  // (false where there is no page)
            codes[i] = __ldg(reinterpret_cast<const uint4*>(pool + (((size_t)fq * Hkv + x.kvh) * P + tk) * D + cch * 16));
        }
      };
      auto store = [&](uint32_t dst, const uint4 (&codes)[NI]) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int rr = 32 * cw + i * RPI + crow;
          uint4 h0, h1;
          codes_half<I8, false>(codes[i].x, h0.x, h0.y);
          codes_half<I8, false>(codes[i].y, h0.z, h0.w);
          codes_half<I8, false>(codes[i].z, h1.x, h1.y);
          codes_half<I8, false>(codes[i].w, h1.z, h1.w);
          sts128(dst + tile_off(rr, 2 * cch), h0);
          sts128(dst + tile_off(rr, 2 * cch + 1), h1);
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      };
      uint4 kc[NI], vc[NI];
      for (int j = 0; j < x.n; ++j, ++it) {
        if ((j & 31) == 0) {
#pragma unroll
          for (int q = 0; q < PW; ++q) {
            const int t = (x.t0 + x.n - 1 - j - lane) * KP + cw * PW + q;
            ph[q] = -1;
            key[q] = kNoKey;
            ks[q] = 0.0f;
            vs[q] = 1.0f;
            if (j + lane < x.n && t < x.sp.T) {
              const int page = x.sp.page(t);
              ph[q] = phys_page(a.c.block_table, x.s.seq, page, a.c.maxp, a.c.nphys, a.c.status);
              if (ph[q] >= 0) {
                key[q] = page * P;
                ks[q] = a.c.k_scale[(size_t)ph[q] * Hkv + x.kvh];
                vs[q] = a.c.v_scale[(size_t)ph[q] * Hkv + x.kvh];
              }
            }
          }
          load(a.c.k_pool, j, kc);
        }
        load(a.c.v_pool, j, vc);
#pragma unroll
        for (int q = 0; q < PW; ++q) {
          const float kk = __shfl_sync(0xffffffffu, ks[q], j & 31);
          const float vv = fmaxf(__shfl_sync(0xffffffffu, vs[q], j & 31), 0x1p-100f);
          const int k0 = __shfl_sync(0xffffffffu, key[q], j & 31);
          if (lane == 0) meta[it & 3][cw * PW + q] = PageMeta{kk, log2f(vv), 1.0f / vv, k0};
        }
        const int sg = it & 1;
        if (it >= 2 && !wait_warp(&k_empty[sg], it / 2 - 1)) {
          ok = false;
          break;
        }
        store(k_sm + sg * TILE, kc);
        mbar_arrive(&k_full[sg]);
        if (j + 1 < x.n && ((j + 1) & 31)) load(a.c.k_pool, j + 1, kc);
        if (it >= 2 && !wait_warp(&v_empty[sg], it / 2 - 1)) {
          ok = false;
          break;
        }
        store(v_sm + sg * TILE, vc);
        mbar_arrive(&v_full[sg]);
      }
      w += x.skip + x.n;
    }
  } else {  // ------------------------------------------------------- products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
    if (warp < 14) {  // a warp a half, one elected thread of it
      const int hf = warp - 12;
      constexpr uint32_t id_qk = instr_desc(kChunkKeys / 2, 0), id_pv = instr_desc(D, 1);
      const uint64_t q_desc = smem_desc(q_sm + hf * TILE, 16, 1024), k_desc = smem_desc(k_sm, 16, 1024);
      const uint64_t v_desc = smem_desc(v_sm, 16384, 1024);
      const uint32_t s_tm = tm + 128 * hf, o_tm = tm + 256 + D * hf;
      int it = 0, p_it = 0;  // tiles so far, and those of this half
      bool ok = true;
      // Columns c of S are there. The pages' facts in `meta` are plain stores of the converters, which this thread has
      // waited for (k_full) and the softmax warps read behind s_full: on a tile's first columns, c = 1, an arrival of
      // its own hands the order on, beside the commit's. (A barrier of the facts' own, waited for by the softmax warps:
      // 1177 -> 1237 us.)
      auto scored = [&](int c) {
        tm_commit(&s_full[hf][c]);
        if (c == 1) mbar_arrive(&s_full[hf][1]);
      };
      auto scores = [&](int c, int sg) {  // (addresses advance in units of 16 bytes)
        const uint64_t k = k_desc + (uint32_t)(sg * (TILE >> 4) + c * 512);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t o = ((i >> 2) * 16384 + (i & 3) * 32) >> 4;
          mma_ss(s_tm + 64 * c, q_desc + o, k + o, id_qk, i > 0);
        }
        scored(c);
      };
      int item = -1;
      if (tid == 384 && w_begin >= w_end) g.cuts[blockIdx.x] = make_int2(-1, 0);
      for (long long w = w_begin, seg = 0; w < w_end && ok; ++seg) {
        const ChunkSeg x = chunk_seg(g, w, w_end, S, n_items, item);
        item = x.item + 1;
        if (tid == 384 && seg == 0) g.cuts[blockIdx.x] = make_int2(x.n > 0 && x.t0 > 0 ? x.item : -1, x.kvh);
        if (x.n == 0) break;
        const bool mine = x.s.count * G - x.rt * kChunkRows > 128 * hf;
        ok = wait_warp(&q_full, (int)seg) && wait_warp(&k_full[it & 1], it / 2);
        if (!ok) break;
        tm_fence_after();
        if (elect_one()) {
          if (mine) {
            scores(1, it & 1);
            scores(0, it & 1);
          }
          tm_commit(&k_empty[it & 1]);  // (a half without rows commits nothing but its word)
        }
        for (int j = 0; j < x.n && ok; ++j, ++it) {
          const int sg = it & 1;
          ok = wait_warp(&v_full[sg], it / 2) && (j + 1 == x.n || wait_warp(&k_full[sg ^ 1], (it + 1) / 2));
          if (mine) {
#pragma unroll 1
            for (int c = 1; c >= 0 && ok; --c) {
              ok = wait_warp(&p_full[hf][c], p_it);
              if (!ok) break;
              tm_fence_after();
              if (elect_one()) {
                const uint64_t v = v_desc + (uint32_t)(sg * (TILE >> 4) + c * 512);
#pragma unroll
                for (int k = 0; k < kChunkKeys / 32; ++k)
                  mma_ts(o_tm, s_tm + 64 * c + 8 * k, v + 128 * k, id_pv, k > 0 || j > 0 || c == 0);
                if (j + 1 < x.n) scores(c, sg ^ 1);
                else scored(c);
              }
            }
            ++p_it;
          }
          if (!ok) break;
          if (elect_one()) {
            tm_commit(&v_empty[sg]);
            if (j + 1 < x.n) tm_commit(&k_empty[sg ^ 1]);
          }
        }
        if (ok && elect_one()) tm_commit(&o_full);
        w += x.skip + x.n;
      }
    }
    __syncwarp();
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  if (warp == 12) tm_free(tm);
  if (tid == 0 && gave_up) raise_flag(a.c.status, ENTMAXKV_DEV_TIMEOUT);
}

// The product kernel for one code type and head dimension, of heads or of pairs of
// them (a translation unit each; one kernel for both cost the capped form 5%: 1179 ->
// 1243 us): the page size and the score forms choose among its variants.
template <bool I8, int D, bool PAIRED>
cudaError_t chunk_run(const ChunkArgs& g, cudaStream_t st);

template <bool I8, int D, int P, bool CAP, bool BIAS, bool PAIRED>
cudaError_t chunk_start(const ChunkArgs& g, cudaStream_t st) {
  const int smem = 6 * kChunkKeys * D * 2 + 1024;
  const cudaError_t e = ensure_smem((const void*)chunk_kernel<I8, D, P, CAP, BIAS, PAIRED>, smem);
  if (e != cudaSuccess) return e;
  return launch_k(true, chunk_kernel<I8, D, P, CAP, BIAS, PAIRED>, dim3(g.blocks), dim3(kChunkThreads), (size_t)smem, st, g);
}
template <bool I8, int D, int P, bool PAIRED>
cudaError_t chunk_form(const ChunkArgs& g, cudaStream_t st) {
  const bool cap = g.a.sc.cap > 0.0f, bias = g.a.sc.slopes != nullptr;
  if (cap) return bias ? chunk_start<I8, D, P, true, true, PAIRED>(g, st) : chunk_start<I8, D, P, true, false, PAIRED>(g, st);
  return bias ? chunk_start<I8, D, P, false, true, PAIRED>(g, st) : chunk_start<I8, D, P, false, false, PAIRED>(g, st);
}
template <bool I8, int D, bool PAIRED>
cudaError_t chunk_pages(const ChunkArgs& g, cudaStream_t st) {
  return g.a.c.P == 32 ? chunk_form<I8, D, 32, PAIRED>(g, st) : chunk_form<I8, D, 16, PAIRED>(g, st);
}

}  // namespace ekv
