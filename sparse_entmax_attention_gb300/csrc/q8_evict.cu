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
// Two launches. The first (a cluster, a thread a slot) decides which slots are
// evicted, and does the books: lengths, free list, the list of what to move. In
// the second a cluster of 8 or 16 blocks has one (slot, KV head) at a time:
//   select  the keep-th largest weight by three counts of 11, 11 and 10 bits of
//           the weights' order-preserving codes, summed over the cluster through
//           distributed shared memory; equal weights by index;
//   move    in place and in one pass: a warp holds one page of the result, K and
//           V, in registers; when all warps of the cluster have loaded theirs (a
//           cluster barrier) they write. Source pages of later pages lie behind
//           all pages written so far, as src(d) ≥ d and src grows.
//
// Bound: the bytes of the weights and the kept codes, and the latency of the
// chain select - barrier - move where few sequences are evicted.
#include "q8_tiles.cuh"

namespace ekv {

constexpr int kEvictPlanThreads = 1024, kEvictPlanBlocks = 8;
constexpr int kEvictWarps = 8, kEvictThreads = kEvictWarps * 32;
constexpr int kEvictKeys = 16384;  // a block's weights that stay in shared memory; more are read again for each count
constexpr int kBins = 2048;

struct EvictItem {
  int seq, L;
};
struct EvictArgs {
  Q8Cache c;
  const int32_t* seq_ids;
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
  int32_t* src;      // [n][Hkv][keep] old key of each kept one
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
  for (int b = me; b < a.n; b += all) {
    const int seq = a.seq_ids[b];
    a.bad[b] = 0;
    if (seq >= 0 && seq < a.c.max_seqs) a.owner[seq] = 0x7fffffff;
  }
  cluster_sync();
  for (int b = me; b < a.n; b += all) {
    const int seq = a.seq_ids[b];
    if (seq >= 0 && seq < a.c.max_seqs) atomicMin(a.owner + seq, b);
  }
  cluster_sync();
  auto slot = [&](int b, uint32_t* st) -> EvictItem {  // L = 0: stays as it is
    EvictItem x{-1, 0};
    if (b >= a.n) return x;
    x.seq = seq_row(a.seq_ids, b, a.c.max_seqs, st);
    if (x.seq < 0) return x;
    if (__ldcg(a.owner + x.seq) != b) {  // named before
      raise_flag(st, ENTMAXKV_DEV_BAD_BATCH);
      return x;
    }
    x.L = seq_len_clamped(a.c.seq_lens, x.seq, a.c.maxp, P, st);
    if (x.L <= a.above || __ldcg(a.bad + b)) x.L = 0;
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
  // pages outside the pool: their slots stay as they are
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
    const EvictItem x = slot(b0 + tid, nullptr);
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

template <bool I8, int D, int P>
__global__ void __launch_bounds__(kEvictThreads, 2) evict_kernel(EvictArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) uint32_t keys_sm[];  // [kEvictKeys]
  __shared__ __align__(16) uint32_t hist[3][kBins];
  __shared__ int sh_scan[32], sh_digit, sh_want;
  __shared__ int warp_more[kEvictWarps], warp_same[kEvictWarps];
  __shared__ __align__(16) int block_cnt[4];  // kept for certain, equal to the edge
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t C;
  asm("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(C));
  const int rank = (int)cluster_rank(), Hkv = a.c.Hkv, keep = a.keep;
  const int n_clusters = gridDim.x / C, take = keep - a.sinks - a.recent;
  const long long n_work = (long long)*a.n_items * Hkv;
  for (long long it = blockIdx.x / C; it < n_work; it += n_clusters) {
    const int item = (int)(it / Hkv), h = (int)(it - (long long)item * Hkv);
    const EvictItem x = a.items[item];
    const int32_t* bt = a.c.block_table + (size_t)x.seq * a.c.maxp;
    int32_t* src = a.src + (size_t)it * keep;
    const int seg = ((x.L + (int)C - 1) / (int)C + 31) / 32 * 32;
    const int lo = min(x.L, rank * seg), hi = min(x.L, lo + seg);
    const int c0 = a.sinks, c1 = x.L - a.recent;  // keys that are chosen among
    auto code = [&](int i) -> uint32_t {  // larger weights have larger codes; NaN the largest, −0 is 0
      const float w = a.w[((size_t)bt[i / P] * Hkv + h) * P + i % P];
      return w != w ? 0xffffffffu : ord_enc(w + 0.0f);
    };
    const bool held = seg <= kEvictKeys;
    uint32_t edge = 0u;
    int want = take;
    if (take > 0) {
      if (held) {
#pragma unroll 8
        for (int i = lo + tid; i < hi; i += kEvictThreads) keys_sm[i - lo] = code(i);
      }
      for (int i = tid; i < 3 * kBins; i += kEvictThreads) (&hist[0][0])[i] = 0u;
      __syncthreads();
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const int shift = p == 0 ? 21 : p == 1 ? 10 : 0;
        const uint32_t mask = p == 2 ? 1023u : 2047u, above = p == 0 ? 0u : 0xffffffffu << (p == 1 ? 21 : 10);
        for (int i = max(lo, c0) + tid; i < min(hi, c1); i += kEvictThreads) {
          const uint32_t k = held ? keys_sm[i - lo] : code(i);
          if (((k ^ edge) & above) == 0u) atomicAdd(&hist[p][k >> shift & mask], 1u);
        }
        cluster_sync();
        // eight bins a thread, the largest codes with the first thread
        uint32_t n8[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        const int bin0 = kBins - 8 - 8 * tid;
        for (int r = 0; r < (int)C; ++r) {
          const uint32_t at = of_block(smem_u32(&hist[p][bin0]), r);
          const uint4 u = ld_cluster4(at), v = ld_cluster4(at + 16);
          n8[0] += u.x, n8[1] += u.y, n8[2] += u.z, n8[3] += u.w;
          n8[4] += v.x, n8[5] += v.y, n8[6] += v.z, n8[7] += v.w;
        }
        int sum = 0, total;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += (int)n8[j];
        int before = block_exclusive_scan(sum, sh_scan, total);
        if (before < want && before + sum >= want) {
#pragma unroll
          for (int j = 7; j >= 0; --j) {
            if (before < want && before + (int)n8[j] >= want) {
              sh_digit = bin0 + j;
              sh_want = want - before;
            }
            before += (int)n8[j];
          }
        }
        __syncthreads();
        edge |= (uint32_t)sh_digit << shift;
        want = sh_want;
        __syncthreads();
      }
    }
    // Each warp has a part of the block's keys: how many are kept for certain and how many equal the edge, then the
    // place of each kept key, the certain ones before it plus the equal ones, of which the first `want` are taken.
    const int wseg = seg / 32 / kEvictWarps + 1, w0 = min(hi, lo + warp * wseg * 32), w1 = min(hi, w0 + wseg * 32);
    auto look = [&](int i, bool& more, bool& same) {
      more = i < w1 && (i < c0 || i >= c1);
      same = false;
      if (i < w1 && !more && take > 0) {
        const uint32_t k = held ? keys_sm[i - lo] : code(i);
        more = k > edge;
        same = k == edge;
      }
    };
    int n_more = 0, n_same = 0;
    for (int i = w0; i < w1; i += 32) {
      bool more, same;
      look(i + lane, more, same);
      n_more += __popc(__ballot_sync(0xffffffffu, more));
      n_same += __popc(__ballot_sync(0xffffffffu, same));
    }
    if (lane == 0) {
      warp_more[warp] = n_more;
      warp_same[warp] = n_same;
    }
    __syncthreads();
    if (tid == 0) {
      int m = 0, s = 0;
      for (int i = 0; i < kEvictWarps; ++i) {
        m += warp_more[i];
        s += warp_same[i];
      }
      block_cnt[0] = m;
      block_cnt[1] = s;
    }
    cluster_sync();
    n_more = n_same = 0;
    for (int r = 0; r < rank; ++r) {
      const uint4 u = ld_cluster4(of_block(smem_u32(block_cnt), r));
      n_more += (int)u.x;
      n_same += (int)u.y;
    }
    for (int i = 0; i < warp; ++i) {
      n_more += warp_more[i];
      n_same += warp_same[i];
    }
    for (int i = w0; i < w1; i += 32) {
      bool more, same;
      look(i + lane, more, same);
      const uint32_t bm = __ballot_sync(0xffffffffu, more), bs = __ballot_sync(0xffffffffu, same);
      const uint32_t below = (1u << lane) - 1u;
      const int m = n_more + __popc(bm & below), s = n_same + __popc(bs & below);
      if (more || (same && s < want)) {
        const int to = m + min(s, want);
        if (to < keep) src[to] = i + lane;
      }
      n_more += __popc(bm);
      n_same += __popc(bs);
    }
    cluster_sync();  // the list is there, and every weight has been read
    constexpr int LPR = D / 16, RPI = 32 / LPR, NI = P / RPI;  // lanes a row, rows a load, loads of a page
    const int pages = (keep + P - 1) / P, wave = (int)C * kEvictWarps;
    const int sub = lane / LPR, ch = lane % LPR;
    for (int j0 = 0; j0 < pages; j0 += wave) {
      const int j = j0 + warp * (int)C + rank, rows = min(P, keep - j * P);
      const int d = j * P + min(lane, rows - 1);
      const bool mine = j < pages;
      int i = mine ? __ldcg(src + d) : 0;
      const bool moves = mine && __shfl_sync(0xffffffffu, i, max(rows, 1) - 1) != j * P + rows - 1;
      uint4 kc[NI], vc[NI];
      float sk = 0.0f, sv = 0.0f, w = 0.0f;
      if (moves) {
        const size_t at = (size_t)bt[i / P] * Hkv + h;  // page and head of the lane's key
        const int off = i % P;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
          const int rl = min(n * RPI + sub, rows - 1);
          const size_t from = (__shfl_sync(0xffffffffu, (unsigned long long)at, rl) * P +
                               __shfl_sync(0xffffffffu, off, rl)) * D + ch * 16;
          kc[n] = __ldcg(reinterpret_cast<const uint4*>(a.c.k_pool + from));
          vc[n] = __ldcg(reinterpret_cast<const uint4*>(a.c.v_pool + from));
        }
        const float k1 = __ldcg(a.c.k_scale + at), v1 = __ldcg(a.c.v_scale + at);
        if (a.w) w = __ldcg(a.w + at * P + off);
        sk = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(k1)));
        sv = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v1)));
        const float rk = __fdiv_rn(k1, sk), rv = __fdiv_rn(v1, sv);
        auto rescale = [&](uint4 (&c)[NI], float ratio) {
          if (!__any_sync(0xffffffffu, ratio != 1.0f)) return;
#pragma unroll
          for (int n = 0; n < NI; ++n) {
            const float r = __shfl_sync(0xffffffffu, ratio, min(n * RPI + sub, rows - 1));
            c[n] = make_uint4(rescale4<I8>(c[n].x, r), rescale4<I8>(c[n].y, r), rescale4<I8>(c[n].z, r),
                              rescale4<I8>(c[n].w, r));
          }
        };
        rescale(kc, rk);
        rescale(vc, rv);
      }
      cluster_sync();
      if (moves) {
        const size_t at = (size_t)bt[j] * Hkv + h;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
          const int t = n * RPI + sub;
          if (t < rows) {
            *reinterpret_cast<uint4*>(a.c.k_pool + (at * P + t) * D + ch * 16) = kc[n];
            *reinterpret_cast<uint4*>(a.c.v_pool + (at * P + t) * D + ch * 16) = vc[n];
          }
        }
        if (lane == 0) {
          a.c.k_scale[at] = sk;
          a.c.v_scale[at] = sv;
        }
        if (a.w && lane < rows) a.w_out[at * P + lane] = w;
      } else if (mine && a.w && a.w_out != a.w && lane < rows) {  // the page stays, its weights are wanted elsewhere
        const size_t at = ((size_t)bt[j] * Hkv + h) * P + lane;
        a.w_out[at] = a.w[at];
      }
    }
    cluster_sync();  // counts and histograms are done with in every block
  }
}

static size_t up256e(size_t x) { return (x + 255) & ~(size_t)255; }

size_t evict_bytes(const entmaxkv_config& cfg, int n, int keep) {
  return up256e((size_t)cfg.max_seqs * 4) + up256e((size_t)n * 4) + up256e((size_t)n * sizeof(EvictItem)) + 256 +
         up256e((size_t)n * cfg.num_kv_heads * keep * 4);
}

template <bool I8, int D, int P>
static cudaError_t evict_t(const EvictArgs& a, int sms, cudaStream_t st) {
  const void* fn = (const void*)evict_kernel<I8, D, P>;
  const int smem = kEvictKeys * 4;
  cudaError_t e = ensure_smem(fn, smem);
  if (e != cudaSuccess) return e;
  const int C = 8;
  // clusters that fit beside one another, two blocks a multiprocessor
  const long long want = (long long)a.n * a.c.Hkv, fit = max(1, 2 * sms / C);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(min(want, fit) * C));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_kernel<I8, D, P>, a);
}
template <bool I8>
static cudaError_t evict_d(const EvictArgs& a, int sms, cudaStream_t st) {
  if (a.c.D == 128) return a.c.P == 32 ? evict_t<I8, 128, 32>(a, sms, st) : evict_t<I8, 128, 16>(a, sms, st);
  return a.c.P == 32 ? evict_t<I8, 64, 32>(a, sms, st) : evict_t<I8, 64, 16>(a, sms, st);
}

cudaError_t launch_evict(const Q8Cache& c, const int32_t* seq_ids, int n, int keep, int above, int sinks, int recent,
                         const float* w, float* w_out, int32_t* lens_out, int32_t* free_pages,
                         const int32_t* free_count, int32_t* count_out, bool i8, void* ws, int sms, cudaStream_t st) {
  EvictArgs a{c, seq_ids, n, keep, above, sinks, recent, w, w_out, lens_out, free_pages, free_count, count_out,
              nullptr, nullptr, nullptr, nullptr, nullptr};
  char* p = static_cast<char*>(ws);
  a.owner = reinterpret_cast<int*>(p);
  p += up256e((size_t)c.max_seqs * 4);
  a.bad = reinterpret_cast<int*>(p);
  p += up256e((size_t)n * 4);
  a.items = reinterpret_cast<EvictItem*>(p);
  p += up256e((size_t)n * sizeof(EvictItem));
  a.n_items = reinterpret_cast<int*>(p);
  p += 256;
  a.src = reinterpret_cast<int32_t*>(p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kEvictPlanBlocks);
  cfg.blockDim = dim3(kEvictPlanThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kEvictPlanBlocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_plan_kernel, a);
  if (e != cudaSuccess) return e;
  return i8 ? evict_d<true>(a, sms, st) : evict_d<false>(a, sms, st);
}

}  // namespace ekv
