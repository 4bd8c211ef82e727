// pages.cu -- block tables, lengths and slot maps of a batch of requests,
// built on the device from a free list.
//
// Slot b's sequence of L tokens grows by n: need = ceil((L+n)/P) − ceil(L/P)
// pages. With the running sums N of the needs and S of the n, a slot is
// admitted while N_b ≤ the list's height, its j-th page is entry
// height − 1 − (N_{b−1} + j) of the list, and its tokens are rows S_{b−1}...
// of the batch. Everything follows from the two sums, so the outputs do not
// depend on the order in which threads run.
//
// Bound: latency, one launch (a decode step of 64 sequences moves 2.3 KB: 6.2 us
// in a graph, of which an empty launch is about 2.5). Every block of a cluster
// scans all slots and then fills its share of the tokens' positions and slots;
// the cluster is there because the reads of lengths end (a cluster barrier)
// before lens_out, which may be seq_lens, is written.
#include "q8.cuh"

namespace ekv {

constexpr int kPlanThreads = 1024;

struct PlanArgs {
  int P, maxp, nphys, max_seqs, n_seqs, total, max_count;
  int32_t* block_table;
  const int32_t* seq_lens;
  uint32_t* status;
  const int32_t* seq_ids;
  const int32_t* n_new;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* lens_out;
  int32_t* start;
  int32_t* count;
  int32_t* positions;
  int64_t* slots;
};

// Exclusive scan of two 64-bit sums over the block.
__device__ __forceinline__ void scan2(long long& a, long long& b, long long (*sh)[2], long long& ta, long long& tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  long long x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    sh[warp][0] = x;
    sh[warp][1] = y;
  }
  __syncthreads();
  if (warp == 0) {
    long long u = lane < nw ? sh[lane][0] : 0, v = lane < nw ? sh[lane][1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long s = __shfl_up_sync(0xffffffffu, u, o), t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) {
        u += s;
        v += t;
      }
    }
    if (lane < nw) {
      sh[lane][0] = u;
      sh[lane][1] = v;
    }
  }
  __syncthreads();
  ta = sh[nw - 1][0];
  tb = sh[nw - 1][1];
  a = (warp ? sh[warp - 1][0] : 0) + x - a;
  b = (warp ? sh[warp - 1][1] : 0) + y - b;
  __syncthreads();
}

// Every block of a cluster takes the slots 1024 at a time, a thread per slot
// for the sums (all blocks the same), then its share of the round's new pages
// and tokens, each thread finding its slot by bisection in the round's sums.
// Lengths and the list's height are written last, by the first block, once the
// whole cluster has read the old ones (they may be the same arrays).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
  pdl_enter();
  __shared__ long long sh[32][2];
  __shared__ int t_end[kPlanThreads], n_end[kPlanThreads];  // running sums of the round, inclusive, from its base
  __shared__ int seq_sh[kPlanThreads], len_sh[kPlanThreads], take_sh[kPlanThreads];
  const int tid = threadIdx.x, P = a.P;
  const int all = gridDim.x * kPlanThreads, me = blockIdx.x * kPlanThreads + tid;  // the grid is one cluster
  const bool head = blockIdx.x == 0;
  uint32_t* status = head ? a.status : nullptr;
  const int fc = min(max(*a.free_count, 0), a.nphys);
  long long t_base = 0, n_base = 0;  // rows and needs of the earlier rounds
  long long used = 0;                // pages handed out
  for (int r0 = 0; r0 < a.n_seqs; r0 += kPlanThreads) {
    const int i = r0 + tid;
    int n = 0, seq = -1, L = 0;
    bool bad = false;
    long long need = 0;
    if (i < a.n_seqs) {
      n = a.n_new[i];
      if (n < 0) {
        raise_flag(status, ENTMAXKV_DEV_BAD_BATCH);
        n = 0;
        bad = true;
      }
      if (n > a.max_count) {  // its rows keep their places, as a refused slot's do
        raise_flag(status, ENTMAXKV_DEV_BAD_BATCH);
        bad = true;
      } else if (n > 0) {
        seq = seq_row(a.seq_ids, i, a.max_seqs, status);
        if (seq >= 0) {
          L = a.seq_lens[seq];
          if (L < 0 || (long long)L + n > (long long)a.maxp * P) {
            raise_flag(status, ENTMAXKV_DEV_CAPACITY);
            bad = true;
          } else {
            need = ((long long)L + n + P - 1) / P - (L + P - 1) / P;
          }
        } else {
          bad = true;
        }
      }
    }
    long long ts = n, ns = need, tt, nt;
    scan2(ts, ns, sh, tt, nt);
    bool ok = !bad;
    if (ok && n > 0 && n_base + ns + need > fc) {
      raise_flag(status, ENTMAXKV_DEV_CAPACITY);
      ok = false;
    }
    if (ok && t_base + ts + n > a.total) {
      raise_flag(status, ENTMAXKV_DEV_BAD_BATCH);
      ok = false;
    }
    if (head && i < a.n_seqs) {
      a.start[i] = (int)min(t_base + ts, 0x7fffffffLL);
      a.count[i] = ok ? n : 0;
    }
    const long long t_left = a.total - t_base;  // rows of the arrays that are left for this round
    t_end[tid] = (int)max(0LL, min(ts + n, t_left));
    n_end[tid] = (int)min(ns + need, 0x7fffffffLL);
    seq_sh[tid] = seq;
    len_sh[tid] = L;
    take_sh[tid] = ok && n > 0;
    __syncthreads();
    // pages: those of the round that the list still holds
    const long long n_fit = max(0LL, min(nt, (long long)fc - n_base));
    for (int j = me; j < n_fit; j += all) {
      int lo = 0, hi = kPlanThreads - 1;
      while (lo < hi) {
        const int m = (lo + hi) >> 1;
        if (n_end[m] > j) hi = m;
        else lo = m + 1;
      }
      if (!take_sh[lo]) continue;
      const int k = j - (lo ? n_end[lo - 1] : 0);
      a.block_table[(size_t)seq_sh[lo] * a.maxp + (len_sh[lo] + P - 1) / P + k] = a.free_pages[fc - 1 - (n_base + j)];
    }
    // tokens
    const int t_fit = (int)max(0LL, min(tt, t_left));
    if (a.positions || a.slots)
      for (int j = me; j < t_fit; j += all) {
        int lo = 0, hi = kPlanThreads - 1;
        while (lo < hi) {
          const int m = (lo + hi) >> 1;
          if (t_end[m] > j) hi = m;
          else lo = m + 1;
        }
        const int k = j - (lo ? t_end[lo - 1] : 0);
        int pos = -1;
        long long slot = -1;
        if (take_sh[lo]) {
          const int L = len_sh[lo], have = (L + P - 1) / P;
          pos = L + k;
          const int lp = pos / P;
          const int ph = lp < have ? a.block_table[(size_t)seq_sh[lo] * a.maxp + lp]
                                   : a.free_pages[fc - 1 - (n_base + (lo ? n_end[lo - 1] : 0) + lp - have)];
          if (ph >= 0 && ph < a.nphys) slot = (long long)ph * P + pos % P;
          else raise_flag(a.status, ENTMAXKV_DEV_BAD_PAGE_TABLE);
        }
        if (a.positions) a.positions[t_base + j] = pos;
        if (a.slots) a.slots[t_base + j] = slot;
      }
    // the admitted needs of the round: those of the slots in front of the first that did not fit
    long long took = take_sh[tid] ? need : 0, dummy = 0, took_all, d_all;
    scan2(took, dummy, sh, took_all, d_all);
    used += took_all;
    t_base += tt;
    n_base += nt;
    __syncthreads();
  }
  // every read of the old lengths and of the list's height is done, in all blocks
  if (gridDim.x > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  }
  if (!head) return;
  if (a.lens_out)
    for (int i = tid; i < a.n_seqs; i += kPlanThreads) {
      const int n = a.count[i];
      if (n > 0) {
        const int seq = a.seq_ids ? a.seq_ids[i] : i;
        a.lens_out[seq] = a.seq_lens[seq] + n;
      }
    }
  if (tid == 0) *a.free_count_out = fc - (int)used;
}

// One block, a sequence after the other: the list's order follows the slots', and a
// sequence named twice is given back once (2.1 us for 4096 tokens, 1.3 us a sequence
// of 2000).
__global__ void __launch_bounds__(kPlanThreads)
    release_kernel(int P, int maxp, int nphys, int max_seqs, int n_seqs, const int32_t* block_table, int32_t* seq_lens,
                   uint32_t* status, const int32_t* seq_ids, int32_t* free_pages, int32_t* free_count) {
  pdl_enter();
  __shared__ int sh[32];
  const int tid = threadIdx.x;
  int fc = min(max(*free_count, 0), nphys);
  for (int i = 0; i < n_seqs; ++i) {
    const int seq = seq_row(seq_ids, i, max_seqs, tid == 0 ? status : nullptr);
    if (seq < 0) continue;
    const int L = seq_len_clamped(seq_lens, seq, maxp, P, tid == 0 ? status : nullptr);
    const int n = (L + P - 1) / P;
    for (int j0 = 0; j0 < n; j0 += kPlanThreads) {
      const int j = j0 + tid;
      int ph = -1;
      if (j < n) ph = phys_page(block_table, seq, n - 1 - j, maxp, nphys, status);
      int total;
      const int at = block_exclusive_scan(ph >= 0 ? 1 : 0, sh, total);
      if (ph >= 0) {
        if (fc + at < nphys) free_pages[fc + at] = ph;
        else raise_flag(status, ENTMAXKV_DEV_CAPACITY);
      }
      fc = min(fc + total, nphys);
    }
    __syncthreads();  // every thread has read this sequence's length
    if (tid == 0) seq_lens[seq] = 0;
    __syncthreads();  // a sequence named twice is empty the second time
  }
  if (tid == 0) *free_count = fc;
}

cudaError_t launch_plan(const entmaxkv_config& cfg, int32_t* block_table, const int32_t* seq_lens, uint32_t* status,
                        const int32_t* seq_ids, const int32_t* n_new, int n_seqs, int total, int max_count,
                        const int32_t* free_pages, const int32_t* free_count, int32_t* free_count_out,
                        int32_t* lens_out, int32_t* start, int32_t* count, int32_t* positions, int64_t* slots,
                        cudaStream_t st) {
  PlanArgs a{cfg.page_size, cfg.max_pages_per_seq, cfg.num_phys_pages, cfg.max_seqs, n_seqs, total, max_count,
             block_table, seq_lens, status, seq_ids, n_new, free_pages, free_count, free_count_out, lens_out, start,
             count, positions, slots};
  // four tokens a thread, up to the eight blocks of a portable cluster (a queue of 333 prompts, 38000 tokens: 11.3 us,
  // 39 with one block; a decode step of 64 sequences has one)
  const int blocks = total > 4 * kPlanThreads ? 8 : total > kPlanThreads ? 2 : 1;
  cudaLaunchConfig_t cfg_l = {};
  cfg_l.gridDim = dim3(blocks);
  cfg_l.blockDim = dim3(kPlanThreads);
  cfg_l.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg_l.attrs = attr;
  cfg_l.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg_l, plan_kernel, a);
}

cudaError_t launch_release(const entmaxkv_config& cfg, const int32_t* block_table, int32_t* seq_lens, uint32_t* status,
                           const int32_t* seq_ids, int n_seqs, int32_t* free_pages, int32_t* free_count,
                           cudaStream_t st) {
  return launch_k(false, release_kernel, dim3(1), dim3(kPlanThreads), 0, st, cfg.page_size, cfg.max_pages_per_seq,
                  cfg.num_phys_pages, cfg.max_seqs, n_seqs, block_table, seq_lens, status, seq_ids, free_pages,
                  free_count);
}

}  // namespace ekv
