// q8_evict.cu -- eviction from the 8-bit paged cache by the weight that keys
// gathered.
//
// A sequence longer than `above` keeps, in each KV head for itself, its first
// `sinks` and last `recent` keys and the heaviest of the others, `keep` in all.
// They move to the front in their order: key d of the shortened sequence is key
// src(d) ≥ d of the old one. A page takes the largest scale s' of the pages its
// keys come from, and a code v becomes nearest(v·r), r = fl32(s/s'), ties to even
// of the exact product, as append rescales. Pages that are left over go back on
// the free list.
//
// plan    (a cluster, a thread a slot) decides which slots are evicted, and does
//         the books: lengths, free list, the list of what to move.
// select  (a block or a cluster for a (slot, KV head)) finds the keep-th largest
//         weight by counts of a few bits at a time of the weights' order-preserving
//         codes, summed over the cluster through distributed shared memory, and
//         lists the kept keys; equal weights go by index.
// move    (a block or a cluster for a (slot, KV head, side)) in place and in one
//         pass: a warp holds one page of the result in registers; when all warps of
//         the cluster have loaded theirs (a cluster barrier) they write. Source pages
//         of later pages lie behind all pages written so far, as src(d) ≥ d and src
//         grows.
// One (slot, KV head) is a chain of latencies (loads, counts, barriers), so they run
// side by side: a block each where they are many or short, clusters of 8 where they
// are few and long. What counts is how many slots are evicted, which the plan finds out: both
// forms are launched, and one returns at once.
//
// Bound: the bytes of the weights and the kept codes, and that chain. Measured (8 KV heads; a launch list, cold):
// plan 7-9 us. One sequence of 131072 tokens to 16384, int8, d = 128 (4 MB of weights, 67 MB of codes in and out):
// select 23 us, of which loads 4, the four counts 11 (half of it cluster barriers) and the listing 5; move 27 us, four
// waves of a load (random rows of 128 bytes), a barrier and a store, 2.5 TB/s. 16 sequences of 1000-32000 to 1024,
// e4m3, d = 64: select 27 us, as long as its longest sequence, move 14 us. All three, int8, d = 128:
// 55 us for 131072 to 16384, 25 for 3000 to 2000, 62 for 32768 to 28000. In one kernel, with K and V in one warp's
// registers and clusters of 16 (of which only a few run at a time), the first took 101 us and the second 160.
#include "q8_tiles.cuh"

namespace ekv {

constexpr int kEvictPlanThreads = 1024, kEvictPlanBlocks = 8;
constexpr int kSelectWarps = 32, kSelectThreads = kSelectWarps * 32;
constexpr int kEvictKeys = 40960;  // a block's weights that stay in shared memory; more are read again for each count
// A block alone counts 11, 11 and 10 bits. A cluster's counts are read by each of its blocks, at about 9 bytes a clock:
// 8 bits at a time (2048 counts of 8 blocks: 7000 clocks a pass; 256: 1000).
constexpr int kBins = 2048;
// Codes of the weights, in their order: NaN above infinity, a key that stays whatever it weighs above all, and a place
// behind the sequence's end below all (minus infinity is 0x007fffff). So the edge is the keep-th largest code.
constexpr uint32_t kCodeStays = 0xffffffffu, kCodeNaN = 0xfffffffeu;
constexpr int kEvictCluster = 8;

struct EvictItem {
  int seq, L;
};
struct EvictArgs {
  Q8Cache c;
  const int32_t* seq_ids;
  const int32_t* count;  // [n] or null: slots with 0 are not looked at
  int n, keep, above, sinks, recent;
  const float* w;
  float* w_out;
  int32_t* lens_out;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* count_out;
  // workspace
  int* owner;        // [max_seqs] the first slot that names a sequence
  int* bad;          // [n] slots with a page outside the pool
  EvictItem* items;  // [n]
  int* n_items;
  uint32_t* src;     // [n][Hkv][keep] where each kept key lies: physical page · page_size + offset
  long long from, to;  // (slot, KV head) pairs to move for which this launch does: from < pairs <= to
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
// The address of the same shared variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t of_block(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint4 ld_cluster4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// The plan for at most 1024 slots, a thread each: what the general form, below, leaves
// in memory between its steps stays in registers and shared memory (one sequence of
// 131k tokens: 7.4 us against 11.3).
__global__ void __launch_bounds__(kEvictPlanThreads) evict_plan_few_kernel(EvictArgs a) {
  pdl_enter();
  __shared__ int sh_scan[32];
  __shared__ int end_sh[kEvictPlanThreads], seq_sh[kEvictPlanThreads], bad_sh[kEvictPlanThreads];
  const int tid = threadIdx.x, P = a.c.P;
  const int all = gridDim.x * kEvictPlanThreads, me = blockIdx.x * kEvictPlanThreads + tid;
  const bool head = blockIdx.x == 0;
  uint32_t* status = head ? a.c.status : nullptr;
  bad_sh[tid] = 0;
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  const int fc = min(max(*a.free_count, 0), a.c.nphys), kept = (a.keep + P - 1) / P;
  int seq = -1, L = 0;
  if (tid < a.n && !(a.count && a.count[tid] == 0)) seq = seq_row(a.seq_ids, tid, a.c.max_seqs, status);
  seq_sh[tid] = seq;
  if (seq >= 0) L = seq_len_clamped(a.c.seq_lens, seq, a.c.maxp, P, status);
  __syncthreads();
  if (seq >= 0) {
    bool before = false;
#pragma unroll 8
    for (int j = 0; j < tid; ++j) before |= seq_sh[j] == seq;
    if (before) {
      raise_flag(status, ENTMAXKV_DEV_BAD_BATCH);
      L = 0;
    }
  }
  if (L <= a.above) L = 0;
  const int have = (L + P - 1) / P;
  int total, at = block_exclusive_scan(have, sh_scan, total);
  end_sh[tid] = at + have;
  __syncthreads();
  auto find = [&](int j) {  // the slot that holds the j-th page
    int lo = 0, hi = kEvictPlanThreads - 1;
    while (lo < hi) {
      const int m = (lo + hi) >> 1;
      if (end_sh[m] > j) hi = m;
      else lo = m + 1;
    }
    return lo;
  };
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
#pragma unroll 4
  for (int j = me; j < total; j += all) {
    const int i = find(j);
    if (phys_page(a.c.block_table, seq_sh[i], j - (i ? end_sh[i - 1] : 0), a.c.maxp, a.c.nphys, a.c.status) < 0)
      for (int r = 0; r < (int)gridDim.x; ++r)  // (every block is told)
        asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(of_block(smem_u32(&bad_sh[i]), r)), "r"(1) : "memory");
  }
  cluster_sync();  // (and every read of the old lengths and of the list's height is done)
  if (bad_sh[tid]) L = 0;
  int items;
  const int item = block_exclusive_scan(L > 0, sh_scan, items), gone = L > 0 ? have - kept : 0;
  at = block_exclusive_scan(gone, sh_scan, total);
  end_sh[tid] = at + gone;
  bad_sh[tid] = have;
  __syncthreads();
#pragma unroll 4
  for (int j = me; j < total; j += all) {
    const int i = find(j), k = j - (i ? end_sh[i - 1] : 0);
    const long long to = (long long)fc + j;
    if (to < a.c.nphys) a.free_pages[to] = a.c.block_table[(size_t)seq_sh[i] * a.c.maxp + bad_sh[i] - 1 - k];
    else raise_flag(a.c.status, ENTMAXKV_DEV_CAPACITY);
  }
  if (!head) return;
  if (L > 0) {
    a.items[item] = EvictItem{seq, L};
    a.lens_out[seq] = a.keep;
  }
  if (tid == 0) {
    *a.n_items = items;
    *a.count_out = min(fc + total, a.c.nphys);
  }
}

// Slots 1024 at a time in every block alike; pages are shared out over the
// cluster. Lengths and the list's height are written last, once all blocks have
// read the old ones (they may be the same arrays).
__global__ void __launch_bounds__(kEvictPlanThreads) evict_plan_kernel(EvictArgs a) {
  pdl_enter();
  __shared__ int sh_scan[32];
  __shared__ int end_sh[kEvictPlanThreads], seq_sh[kEvictPlanThreads], have_sh[kEvictPlanThreads];
  const int tid = threadIdx.x, P = a.c.P;
  const int all = gridDim.x * kEvictPlanThreads, me = blockIdx.x * kEvictPlanThreads + tid;
  const bool head = blockIdx.x == 0;
  uint32_t* status = head ? a.c.status : nullptr;
  const int fc = min(max(*a.free_count, 0), a.c.nphys), kept = (a.keep + P - 1) / P;
  auto idle = [&](int b) { return a.count && a.count[b] == 0; };
  for (int b = me; b < a.n; b += all) {
    const int seq = idle(b) ? -1 : a.seq_ids[b];
    a.bad[b] = 0;
    if (seq >= 0 && seq < a.c.max_seqs) a.owner[seq] = 0x7fffffff;
  }
  cluster_sync();
  for (int b = me; b < a.n; b += all) {
    const int seq = idle(b) ? -1 : a.seq_ids[b];
    if (seq >= 0 && seq < a.c.max_seqs) atomicMin(a.owner + seq, b);
  }
  cluster_sync();
  auto slot = [&](int b, uint32_t* st) -> EvictItem {  // L = 0: stays as it is
    EvictItem x{-1, 0};
    if (b >= a.n || idle(b)) return x;
    x.seq = seq_row(a.seq_ids, b, a.c.max_seqs, st);
    if (x.seq < 0) return x;
    if (__ldcg(a.owner + x.seq) != b) {  // named before
      raise_flag(st, ENTMAXKV_DEV_BAD_BATCH);
      return x;
    }
    x.L = seq_len_clamped(a.c.seq_lens, x.seq, a.c.maxp, P, st);
    if (x.L <= a.above) x.L = 0;
    return x;
  };
  auto find = [&](int j) {  // the round's slot that holds its j-th page
    int lo = 0, hi = kEvictPlanThreads - 1;
    while (lo < hi) {
      const int m = (lo + hi) >> 1;
      if (end_sh[m] > j) hi = m;
      else lo = m + 1;
    }
    return lo;
  };
  // Pages outside the pool: their slots stay as they are. Each block numbers a round's pages for itself and looks at its
  // share, so the marks are read behind the barrier only: a block that saw another's would number fewer.
  for (int b0 = 0; b0 < a.n; b0 += kEvictPlanThreads) {
    const EvictItem x = slot(b0 + tid, status);
    const int pages = (x.L + P - 1) / P;
    int total;
    const int at = block_exclusive_scan(pages, sh_scan, total);
    end_sh[tid] = at + pages;
    seq_sh[tid] = x.seq;
    __syncthreads();
    for (int j = me; j < total; j += all) {
      const int i = find(j);
      if (phys_page(a.c.block_table, seq_sh[i], j - (i ? end_sh[i - 1] : 0), a.c.maxp, a.c.nphys, a.c.status) < 0)
        a.bad[b0 + i] = 1;
    }
    __syncthreads();
  }
  cluster_sync();
  int items = 0;
  long long freed = 0;
  for (int b0 = 0; b0 < a.n; b0 += kEvictPlanThreads) {
    EvictItem x = slot(b0 + tid, nullptr);
    if (x.L > 0 && __ldcg(a.bad + b0 + tid)) x.L = 0;
    int some, total;
    const int at_item = block_exclusive_scan(x.L > 0, sh_scan, some);
    if (head && x.L > 0) a.items[items + at_item] = x;
    const int have = (x.L + P - 1) / P, gone = x.L > 0 ? have - kept : 0;
    const int at = block_exclusive_scan(gone, sh_scan, total);
    end_sh[tid] = at + gone;
    seq_sh[tid] = x.seq;
    have_sh[tid] = have;
    __syncthreads();
    for (int j = me; j < total; j += all) {
      const int i = find(j), k = j - (i ? end_sh[i - 1] : 0);
      const long long to = fc + freed + j;
      if (to < a.c.nphys) a.free_pages[to] = a.c.block_table[(size_t)seq_sh[i] * a.c.maxp + have_sh[i] - 1 - k];
      else raise_flag(a.c.status, ENTMAXKV_DEV_CAPACITY);
    }
    items += some;
    freed += total;
    __syncthreads();
  }
  cluster_sync();
  if (!head) return;
  for (int i = tid; i < items; i += kEvictPlanThreads) a.lens_out[a.items[i].seq] = a.keep;
  if (tid == 0) {
    *a.n_items = items;
    *a.count_out = (int)min(fc + freed, (long long)a.c.nphys);
  }
}

// Codes times r ≤ 1, rounded once from the exact product, ties to even.
template <bool I8>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
  if constexpr (I8) {
    // 2^23 + 128 + v as a float for each byte; v·r + 1.5·2^23 is rounded to a whole number by one FMA
    const uint32_t u = w ^ 0x80808080u;
    const unsigned long long off = f2_splat(-8388736.0f), mg = f2_splat(12582912.0f), r2 = f2_splat(r);
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float f0 = __uint_as_float(__byte_perm(u, 0x4b000000u, j ? 0x7442 : 0x7440));
      const float f1 = __uint_as_float(__byte_perm(u, 0x4b000000u, j ? 0x7443 : 0x7441));
      float y0, y1;
      f2_unpack(f2_fma(f2_add(f2_pack(f0, f1), off), r2, mg), y0, y1);
      q[2 * j] = __float_as_uint(y0);
      q[2 * j + 1] = __float_as_uint(y1);
    }
    return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
  } else {
    uint32_t h[2], out = 0u;
    e4m3x4_half(w, h[0], h[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      // towards zero, with the last bit set where that is not exact: rounding this to four bits rounds once
      float y0 = __fmul_rz(v.x, r), y1 = __fmul_rz(v.y, r);
      if (fmaf(v.x, r, -y0) != 0.0f) y0 = __uint_as_float(__float_as_uint(y0) | 1u);
      if (fmaf(v.y, r, -y1) != 0.0f) y1 = __uint_as_float(__float_as_uint(y1) | 1u);
      uint16_t c;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(c) : "f"(y1), "f"(y0));
      out |= (uint32_t)c << (16 * j);
    }
    return out;
  }
}

// The launch's block or cluster count, and whether it is this form's turn.
struct EvictTurn {
  int C, rank, first, step;
  long long n_work;
  bool mine;
};
__device__ __forceinline__ EvictTurn evict_turn(const EvictArgs& a, int sides) {
  uint32_t size;
  asm("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(size));
  EvictTurn t;
  t.C = (int)size;
  t.rank = (int)cluster_rank();
  t.first = blockIdx.x / t.C;
  t.step = gridDim.x / t.C;
  const long long pairs = (long long)*a.n_items * a.c.Hkv;
  t.n_work = pairs * sides;
  t.mine = pairs > a.from && pairs <= a.to;
  return t;
}
__device__ __forceinline__ void evict_sync(int C) {
  if (C > 1) cluster_sync();
  else __syncthreads();
}

template <int P>
__global__ void __launch_bounds__(kSelectThreads, 1) evict_select_kernel(EvictArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) uint32_t keys_sm[];  // [kEvictKeys]
  __shared__ __align__(16) uint32_t hist[3 * kBins];
  __shared__ int sh_scan[32], sh_digit, sh_want;
  __shared__ int warp_more[kSelectWarps], warp_same[kSelectWarps];
  __shared__ __align__(16) int block_cnt[4];  // kept for certain, equal to the edge
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hkv = a.c.Hkv, keep = a.keep;
  const EvictTurn turn = evict_turn(a, 1);
  if (!turn.mine) return;
  const int C = turn.C, rank = turn.rank;
  for (long long it = turn.first; it < turn.n_work; it += turn.step) {
    const int item = (int)(it / Hkv), h = (int)(it - (long long)item * Hkv);
    const EvictItem x = a.items[item];
    const int32_t* bt = a.c.block_table + (size_t)x.seq * a.c.maxp;
    uint32_t* src = a.src + (size_t)it * keep;
    const int seg = ((x.L + C - 1) / C + 127) / 128 * 128;
    const int lo = min(x.L, rank * seg), hi = min(x.L, lo + seg);
    auto codes_at = [&](int i) -> uint4 {  // of four keys, the first a multiple of 4
      float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (a.w) w = *reinterpret_cast<const float4*>(a.w + ((size_t)bt[i / P] * Hkv + h) * P + i % P);
      const float v[4] = {w.x, w.y, w.z, w.w};
      uint32_t k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        k[j] = v[j] != v[j] ? kCodeNaN : ord_enc(v[j] + 0.0f);  // (−0 is 0)
        if (i + j < a.sinks || i + j >= x.L - a.recent) k[j] = i + j < x.L ? kCodeStays : 0u;
      }
      return make_uint4(k[0], k[1], k[2], k[3]);
    };
    const bool held = seg <= kEvictKeys;
    auto codes = [&](int i) -> uint4 { return held ? *reinterpret_cast<const uint4*>(keys_sm + i - lo) : codes_at(i); };
    if (held) {
#pragma unroll 8
      for (int i = lo + 4 * tid; i < hi; i += 4 * kSelectThreads) *reinterpret_cast<uint4*>(keys_sm + i - lo) = codes_at(i);
    }
    uint32_t edge = 0u;
    int want = keep;
    const int bits = C > 1 ? 8 : 11, bins = 1 << bits, passes = C > 1 ? 4 : 3;
    for (int i = tid; i < passes * bins; i += kSelectThreads) hist[i] = 0u;
    __syncthreads();
#pragma unroll 1
    for (int p = 0; p < passes; ++p) {
      const int shift = max(0, 32 - bits * (p + 1));
      const uint32_t mask = C == 1 && p == 2 ? 1023u : (uint32_t)bins - 1u, above = p ? 0xffffffffu << (32 - bits * p) : 0u;
      uint32_t* count = hist + p * bins;
#pragma unroll 4
      for (int i = lo + 4 * tid; i < hi; i += 4 * kSelectThreads) {
        const uint4 k = codes(i);
        if (((k.x ^ edge) & above) == 0u) atomicAdd(count + (k.x >> shift & mask), 1u);
        if (((k.y ^ edge) & above) == 0u) atomicAdd(count + (k.y >> shift & mask), 1u);
        if (((k.z ^ edge) & above) == 0u) atomicAdd(count + (k.z >> shift & mask), 1u);
        if (((k.w ^ edge) & above) == 0u) atomicAdd(count + (k.w >> shift & mask), 1u);
      }
      evict_sync(C);
      // four bins a thread, the largest codes with the first thread
      uint32_t n4[4] = {0u, 0u, 0u, 0u};
      const int bin0 = bins - 4 - 4 * tid;
      if (bin0 >= 0) {
        uint4 u[kEvictCluster];  // (all blocks' counts in flight)
#pragma unroll
        for (int r = 0; r < kEvictCluster; ++r)
          u[r] = r < C ? ld_cluster4(of_block(smem_u32(count + bin0), r)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int r = 0; r < kEvictCluster; ++r) n4[0] += u[r].x, n4[1] += u[r].y, n4[2] += u[r].z, n4[3] += u[r].w;
      }
      const int sum = (int)(n4[0] + n4[1] + n4[2] + n4[3]);
      int total, before = block_exclusive_scan(sum, sh_scan, total);
      if (before < want && before + sum >= want) {
#pragma unroll
        for (int j = 3; j >= 0; --j) {
          if (before < want && before + (int)n4[j] >= want) {
            sh_digit = bin0 + j;
            sh_want = want - before;
          }
          before += (int)n4[j];
        }
      }
      __syncthreads();
      edge |= (uint32_t)sh_digit << shift;
      want = sh_want;
      __syncthreads();
    }
    // Each warp has a part of the block's keys, four of them a lane at a time: how many lie above the edge and how many
    // equal it, then the place of each kept key, those above before it plus the equal ones, of which the first `want`
    // are taken.
    const int wseg = (seg / 128 + kSelectWarps - 1) / kSelectWarps * 128;
    const int w0 = min(hi, lo + warp * wseg), w1 = min(hi, w0 + wseg);
    int n_more = 0, n_same = 0;
#pragma unroll 2
    for (int i = w0 + 4 * lane; i < w1; i += 128) {
      const uint4 k = codes(i);
      n_more += (int)(k.x > edge) + (int)(k.y > edge) + (int)(k.z > edge) + (int)(k.w > edge);
      n_same += (int)(k.x == edge) + (int)(k.y == edge) + (int)(k.z == edge) + (int)(k.w == edge);
    }
    n_more = __reduce_add_sync(0xffffffffu, n_more);
    n_same = __reduce_add_sync(0xffffffffu, n_same);
    const bool ties = n_same > 0;  // among the warp's own keys
    if (lane == 0) {
      warp_more[warp] = n_more;
      warp_same[warp] = n_same;
    }
    __syncthreads();
    if (warp == 0) {
      const int m = __reduce_add_sync(0xffffffffu, lane < kSelectWarps ? warp_more[lane] : 0);
      const int n = __reduce_add_sync(0xffffffffu, lane < kSelectWarps ? warp_same[lane] : 0);
      if (lane == 0) {
        block_cnt[0] = m;
        block_cnt[1] = n;
      }
    }
    evict_sync(C);
    {  // those of the blocks and of the warps in front
      uint4 u = make_uint4(0u, 0u, 0u, 0u);
      if (lane < rank) u = ld_cluster4(of_block(smem_u32(block_cnt), lane));
      n_more = __reduce_add_sync(0xffffffffu, (int)u.x + (lane < warp ? warp_more[lane] : 0));
      n_same = __reduce_add_sync(0xffffffffu, (int)u.y + (lane < warp ? warp_same[lane] : 0));
    }
    for (int i0 = w0; i0 < w1; i0 += 1024) {
      int page[1024 / P / 32];  // of the next 1024 keys, as the table has them
#pragma unroll
      for (int q = 0; q < 1024 / P / 32; ++q) page[q] = i0 / P + 32 * q + lane <= (x.L - 1) / P ? bt[i0 / P + 32 * q + lane] : 0;
      const int i1 = min(w1, i0 + 1024);
      for (int i = i0 + 4 * lane; i - 4 * lane < i1; i += 128) {
        const uint4 k4 = i < i1 ? codes(i) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        const int at = (i - i0) / P;
        int ph = __shfl_sync(0xffffffffu, page[0], at & 31);
        if (P == 16) {
          const int ph1 = __shfl_sync(0xffffffffu, page[1024 / P / 32 - 1], at & 31);
          if (at >= 32) ph = ph1;
        }
        const uint32_t place = (uint32_t)ph * P + i % P, below = (1u << lane) - 1u;
        int m = n_more, n = n_same;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t more = __ballot_sync(0xffffffffu, k[j] > edge);
          m += __popc(more & below);
          n_more += __popc(more);
        }
        if (ties) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t same = __ballot_sync(0xffffffffu, k[j] == edge);
            n += __popc(same & below);
            n_same += __popc(same);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int to = m + min(n, want);
          if ((k[j] > edge || (ties && k[j] == edge && n < want)) && to < keep) src[to] = place + j;
          m += k[j] > edge;
          if (ties) n += k[j] == edge;
        }
      }
    }
    evict_sync(C);  // counts and histograms are done with in every block
  }
}

template <bool I8, int D, int P>
__global__ void __launch_bounds__(1024, 1) evict_move_kernel(EvictArgs a) {
  pdl_enter();
  constexpr int LPR = D / 16, RPI = 32 / LPR, NI = P / RPI;  // lanes a row, rows a load, loads of a page
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, Hkv = a.c.Hkv, keep = a.keep;
  const EvictTurn turn = evict_turn(a, 2);
  if (!turn.mine) return;
  const int pages = (keep + P - 1) / P, wave = turn.C * (blockDim.x >> 5);
  const int sub = lane / LPR, ch = lane % LPR;
  for (long long it = turn.first; it < turn.n_work; it += turn.step) {
    const long long pair = it >> 1;
    const int side = (int)(it & 1), item = (int)(pair / Hkv), h = (int)(pair - (long long)item * Hkv);
    const int32_t* bt = a.c.block_table + (size_t)a.items[item].seq * a.c.maxp;
    const uint32_t* src = a.src + (size_t)pair * keep;
    uint8_t* pool = side ? a.c.v_pool : a.c.k_pool;
    float* scales = side ? a.c.v_scale : a.c.k_scale;
    const bool weighs = a.w && !side;
    auto list = [&](int j) -> uint32_t {  // where the lane's key of page j lies
      return j < pages ? src[j * P + min(lane, min(P, keep - j * P) - 1)] : 0u;
    };
    int j = warp * turn.C + turn.rank;
    uint32_t next = list(j);
    for (int j0 = 0; j0 < pages; j0 += wave, j += wave) {
      const int rows = min(P, keep - j * P);
      const bool mine = j < pages;
      const uint32_t t = next;
      const size_t to = mine ? (size_t)bt[j] * Hkv + h : 0;
      next = list(j + wave);
      // (a key that lies where it should has all before it in their places)
      const bool moves = mine && __shfl_sync(0xffffffffu, t, max(rows, 1) - 1) != (uint32_t)bt[mine ? j : 0] * P + rows - 1;
      uint4 codes[NI];
      float top = 0.0f, w = 0.0f;
      if (moves) {
        const size_t at = (size_t)(t / P) * Hkv + h;  // page and head of the lane's key
        const size_t key = at * P + t % P;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
          const size_t from = __shfl_sync(0xffffffffu, (unsigned long long)key, min(n * RPI + sub, rows - 1)) * D + ch * 16;
          codes[n] = __ldcg(reinterpret_cast<const uint4*>(pool + from));
        }
        const float own = __ldcg(scales + at);
        if (weighs) w = __ldcg(a.w + key);
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(own)));
        const float ratio = own == top ? 1.0f : __fdiv_rn(own, top);  // (0/0 of pages that hold nothing but zeros)
        if (__any_sync(0xffffffffu, ratio != 1.0f)) {
#pragma unroll
          for (int n = 0; n < NI; ++n) {
            const float r = __shfl_sync(0xffffffffu, ratio, min(n * RPI + sub, rows - 1));
            codes[n] = make_uint4(rescale4<I8>(codes[n].x, r), rescale4<I8>(codes[n].y, r), rescale4<I8>(codes[n].z, r),
                                  rescale4<I8>(codes[n].w, r));
          }
        }
      }
      if (j + wave < pages && lane < P) {  // the next wave's keys on their way, beside the barrier and the stores
        const size_t key = ((size_t)(next / P) * Hkv + h) * P + next % P;
        asm volatile("prefetch.global.L2 [%0];\n" ::"l"(pool + key * D));
      }
      evict_sync(turn.C);
      if (moves) {
#pragma unroll
        for (int n = 0; n < NI; ++n) {
          const int row = n * RPI + sub;
          if (row < rows) *reinterpret_cast<uint4*>(pool + (to * P + row) * D + ch * 16) = codes[n];
        }
        if (lane == 0) scales[to] = top;
        if (weighs && lane < rows) a.w_out[to * P + lane] = w;
      } else if (mine && weighs && a.w_out != a.w && lane < rows) {  // the page stays, its weights are wanted elsewhere
        a.w_out[to * P + lane] = a.w[to * P + lane];
      }
    }
  }
}

static size_t up256e(size_t x) { return (x + 255) & ~(size_t)255; }

size_t evict_bytes(const entmaxkv_config& cfg, int n, int keep) {
  return up256e((size_t)cfg.max_seqs * 4) + up256e((size_t)n * 4) + up256e((size_t)n * sizeof(EvictItem)) + 256 +
         up256e((size_t)n * cfg.num_kv_heads * keep * 4);
}

static cudaError_t evict_launch(void (*kernel)(EvictArgs), const EvictArgs& a, long long clusters, int C, int threads,
                                int smem, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * C));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool I8, int D, int P>
static cudaError_t evict_t(EvictArgs a, int sms, cudaStream_t st) {
  // Pairs up to which each has a cluster. A block alone takes as long as its pages do, whatever runs beside it; clusters
  // run about 16 at a time. Measured, clusters/blocks alone, int8, d = 128, 8, 16, 24 and 32 pairs: 2400 to 2048 tokens
  // 27/31, 37/31, 39/31, 51/31 us; 4700 to 4096 29/44, 41/45, 43/45, 56/45; 9000 to 8000 35/68, 45/70, 55/70, 69/72; 17000
  // to 16000 43/111, 57/117, 85/121, 101/125; 32000 to 1024 27/39, 39/39, 43/39, 53/39. Launching both costs 2 us.
  // The rule knows what the move depends on, pairs and keys that stay. The selection goes by the old length, which only
  // the device knows: 16 pairs of 131072 to 1024 are blocks alone, whose weights do not fit (158 us, 8 pairs 44).
  const long long most = (long long)a.n * a.c.Hkv, few = min(sms / 4, max(8, a.keep / 160));
  const int smem = kEvictKeys * 4;
  cudaError_t e = ensure_smem((const void*)evict_select_kernel<P>, smem);
  for (int step = 0; step < 2; ++step) {  // select, move
    if (e == cudaSuccess) {
      a.from = 0;
      a.to = few;
      e = step ? evict_launch(evict_move_kernel<I8, D, P>, a, min(2 * min(most, few), sms / 4LL), kEvictCluster, 512, 0, st)
               : evict_launch(evict_select_kernel<P>, a, min(min(most, few), sms / 8LL), kEvictCluster, kSelectThreads, smem, st);
    }
    if (most > few && e == cudaSuccess) {
      a.from = few;
      a.to = most;
      e = step ? evict_launch(evict_move_kernel<I8, D, P>, a, min(2 * most, 4LL * sms), 1, 512, 0, st)
               : evict_launch(evict_select_kernel<P>, a, min(most, (long long)sms), 1, kSelectThreads, smem, st);
    }
  }
  return e;
}
template <bool I8>
static cudaError_t evict_d(const EvictArgs& a, int sms, cudaStream_t st) {
  if (a.c.D == 128) return a.c.P == 32 ? evict_t<I8, 128, 32>(a, sms, st) : evict_t<I8, 128, 16>(a, sms, st);
  return a.c.P == 32 ? evict_t<I8, 64, 32>(a, sms, st) : evict_t<I8, 64, 16>(a, sms, st);
}

cudaError_t launch_evict(const Q8Cache& c, const int32_t* seq_ids, const int32_t* count, int n, int keep, int above, int sinks, int recent,
                         const float* w, float* w_out, int32_t* lens_out, int32_t* free_pages,
                         const int32_t* free_count, int32_t* count_out, bool i8, void* ws, int sms, cudaStream_t st) {
  EvictArgs a{c, seq_ids, count, n, keep, above, sinks, recent, w, w_out, lens_out, free_pages, free_count, count_out,
              nullptr, nullptr, nullptr, nullptr, nullptr, 0, 0};
  char* p = static_cast<char*>(ws);
  a.owner = reinterpret_cast<int*>(p);
  p += up256e((size_t)c.max_seqs * 4);
  a.bad = reinterpret_cast<int*>(p);
  p += up256e((size_t)n * 4);
  a.items = reinterpret_cast<EvictItem*>(p);
  p += up256e((size_t)n * sizeof(EvictItem));
  a.n_items = reinterpret_cast<int*>(p);
  p += 256;
  a.src = reinterpret_cast<uint32_t*>(p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kEvictPlanBlocks);
  cfg.blockDim = dim3(kEvictPlanThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kEvictPlanBlocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, n <= kEvictPlanThreads ? evict_plan_few_kernel : evict_plan_kernel, a);
  if (e != cudaSuccess) return e;
  return i8 ? evict_d<true>(a, sms, st) : evict_d<false>(a, sms, st);
}

}  // namespace ekv
