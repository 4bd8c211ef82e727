// q8_weigh_chunk.cu -- the list of slots, row tiles and segments, and the
// launches of the weights of many rows (q8_weigh_chunk.cuh).
#include "q8_weigh_chunk.cuh"

namespace ekv {

template <>
cudaError_t weigh_chunk_run<true, 128>(const WcArgs& g, cudaStream_t st);
template <>
cudaError_t weigh_chunk_run<true, 64>(const WcArgs& g, cudaStream_t st);
template <>
cudaError_t weigh_chunk_run<false, 128>(const WcArgs& g, cudaStream_t st);
template <>
cudaError_t weigh_chunk_run<false, 64>(const WcArgs& g, cudaStream_t st);

// One block: slots 1024 at a time, then the round's row tiles, a thread each;
// when all key tiles are counted, the shares of the rows and the segments.
__global__ void __launch_bounds__(1024) weigh_plan_kernel(WcArgs g) {
  pdl_enter();
  __shared__ int sh_scan[32];
  __shared__ int end_sh[1024], lo_sh[1024];
  __shared__ unsigned long long all_sh;
  const Q8WeighArgs& a = g.a;
  const int tid = threadIdx.x, P = a.c.P, G = a.c.G, n = a.b.n_seqs;
  if (tid == 0) all_sh = 0ull;
  int tiles = 0;
  for (int b0 = 0; b0 < n; b0 += 1024) {
    const int b = b0 + tid;
    Q8Slot s{-1, 0, 0, 0};
    if (b < n) s = q8_slot(a.c, a.b, b, a.c.status);
    int nrt = (int)(((long long)s.count * G + kWcRows - 1) / kWcRows), total;
    const int at = block_exclusive_scan(nrt, sh_scan, total);
    end_sh[tid] = at + nrt;
    lo_sh[tid] = 0x7fffffff;
    __syncthreads();
    for (int j = tid; j < total; j += 1024) {
      int lo = 0, hi = 1023;
      while (lo < hi) {
        const int m = (lo + hi) >> 1;
        if (end_sh[m] > j) hi = m;
        else lo = m + 1;
      }
      const int rt = j - (lo ? end_sh[lo - 1] : 0);
      const Q8Slot q = q8_slot(a.c, a.b, b0 + lo, nullptr);
      const int t0 = rt * kWcRows / G, t1 = min(q.count, (rt * kWcRows + kWcRows - 1) / G + 1);
      const int x0 = q.L - q.count;
      WcRows r{x0 + t0, x0 + t1 - 1, 0x7fffffff, 0};
      const int w = a.sc.window;
      if (a.sc.first_key) {
#pragma unroll 4
        for (int i = t0; i < t1; ++i) {
          const int first = max(a.sc.first_key[q.start + i], w > 0 ? max(0, x0 + i - w + 1) : 0);
          // (a row that sees nothing of its own bounds no key)
          if (first <= x0 + i) r.lo_min = min(r.lo_min, first);
          r.lo_max = max(r.lo_max, first);
        }
      } else {
        r.lo_min = w > 0 ? max(0, r.pos_min - w + 1) : 0;
        r.lo_max = w > 0 ? max(0, r.pos_max - w + 1) : 0;
      }
      atomicMin(&lo_sh[lo], r.lo_min);
      if (tiles + j < g.max_tiles) {
        g.rows[tiles + j] = r;
        g.slot_of[tiles + j] = b0 + lo;
      }
    }
    __syncthreads();
    if (b < n) {
      if (nrt > 0 && tiles + at + nrt > g.max_tiles) {  // rows that several slots claim: past the list
        raise_flag(a.c.status, ENTMAXKV_DEV_BAD_BATCH);
        nrt = 0;
      }
      WcSlot x{};
      if (nrt > 0) {
        x = WcSlot{s.seq, s.L, s.start, s.count};
        x.pre = a.sc.prefix ? min(max(a.sc.prefix[b], 0), s.L) : 0;
        x.npages = (s.L + P - 1) / P;
        x.wfirst = lo_sh[tid] >= s.L ? x.npages : lo_sh[tid] / P;
        x.npre = min((x.pre + P - 1) / P, x.wfirst);
        x.fresh = s.L - min(max(a.fresh ? a.fresh[b] : s.count, 0), s.L);
        x.lwfirst = a.decay != 1.0f ? 0 : min(x.wfirst, x.fresh / P);
        x.lnpre = min(x.npre, x.lwfirst);
        x.T = (int)(((long long)(x.lnpre + x.npages - x.lwfirst) * P + kWcKeys - 1) / kWcKeys);
        x.nrt = nrt;
        x.rt0 = tiles + at;
        atomicAdd(&all_sh, (unsigned long long)x.T * a.c.Hkv);
      }
      g.slots[b] = x;
    }
    tiles = min(tiles + total, g.max_tiles);  // (rows claimed over and over: the sum may pass 31 bits)
    __syncthreads();
  }
  // rows are shared out where key tiles alone give a block less than kWcTurns segments
  const unsigned long long all = all_sh, want = (unsigned long long)kWcTurns * g.blocks;
  const int shares = all > 0 && all < want ? (int)((want + all - 1) / all) : 1;
  __shared__ long long sum_sh[32];
  long long base = 0;
  for (int b0 = 0; b0 < n; b0 += 1024) {
    const int b = b0 + tid, lane = tid & 31, warp = tid >> 5;
    long long mine = 0;
    if (b < n) {
      const int nrt = g.slots[b].nrt, split = max(1, min(nrt, shares));
      g.slots[b].nsplit = split;
      mine = (long long)g.slots[b].T * a.c.Hkv * split;
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) sum_sh[warp] = inc;
    __syncthreads();
    long long at = base + inc - mine;
    for (int i = 0; i < 32; ++i) {
      if (i < warp) at += sum_sh[i];
      base += sum_sh[i];
    }
    if (b < n) g.cum[b] = at;
    __syncthreads();
  }
  if (tid == 0) {
    g.cum[n] = base;
    *g.n_tiles = tiles;
  }
  if (shares > 1)
    for (long long i = tid; i < 8 * base; i += 1024) g.done[i] = 0;
}

// Eight bf16 values times a power of two as halves.
__device__ __forceinline__ uint4 halves_of(const uint4& v, float scale) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(__uint_as_float(w[i] << 16) * scale, __uint_as_float(w[i] & 0xffff0000u) * scale);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The rows of a (row tile, KV head) as the products want them, and what the sums
// know of them: a block of 128 threads, a row each for the facts, D/8 threads a
// row for the copy. Rows that add nothing are laid out as zeros.
template <int D>
__global__ void __launch_bounds__(128) weigh_pack_kernel(WcArgs g) {
  pdl_enter();
  const Q8WeighArgs& a = g.a;
  const int kvh = blockIdx.y, tid = threadIdx.x, G = a.c.G, Hkv = a.c.Hkv;
  __shared__ long long at_sh[kWcRows];
  __shared__ uint32_t top_sh[4];
  for (int tile = blockIdx.x; tile < g.max_tiles; tile += gridDim.x) {
    if (tile >= *g.n_tiles) return;
    const WcSlot s = g.slots[g.slot_of[tile]];
    const int rt = tile - s.rt0;
    if (rt >= s.nrt) return;  // (of a slot past the list)
    const int left = s.count * G - rt * kWcRows, rho = rt * kWcRows + tid;
    const bool mine = tid < left;
    const int tok = mine ? rho / G : 0, head = kvh * G + (mine ? rho - tok * G : 0);
    const long long row = s.start + tok;
    const size_t to = (size_t)kvh * g.max_tiles + tile;
    WcFacts& f = g.facts[to];
    const int first = rt * kWcRows / G, pos = s.L - s.count + tok, pos0 = s.L - s.count + first;
    float c = 0.0f, slope = 0.0f;
    int lo = 0;
    bool counts = false;
    if (mine) {
      const float tau = a.tau[row * Hkv * G + head], coef = a.coef ? a.coef[row * Hkv * G + head] : 1.0f;
      counts = fabsf(tau) < CUDART_INF_F && coef > 0.0f;
      if (a.sc.slopes) slope = -a.sc.slopes[head] * kLog2e;
      if (a.sc.first_key) lo = a.sc.first_key[row];
      if (counts) c = a.coef ? fmaf(-tau, kLog2e, __log2f(coef)) : -tau * kLog2e;
    }
    at_sh[tid] = counts ? row * a.q.ts + (long long)head * a.q.hs : -1;
    const float ahead = (float)(pos - pos0);
    f.c[tid] = c;
    f.near[tid] = fmaf(slope, ahead, c);
    f.slope[tid] = slope;
    f.ahead[tid] = ahead;
    f.lo[tid] = lo;
    const uint32_t some = __ballot_sync(0xffffffffu, counts);
    if ((tid & 31) == 0) f.counts[tid >> 5] = some;
    const int whole = __syncthreads_and(counts);
    if (tid == 0) {
      f.pos0 = pos0;
      f.skip = rt * kWcRows - first * G;
      f.whole = whole;
    }
    constexpr int CPR = D / 8, N = kWcRows * CPR / 128;
    uint4 v[N];
    uint32_t top = 0u;  // of the finite magnitudes, two at a time
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int rl = (i * 128 + tid) / CPR, ch = (i * 128 + tid) % CPR;
      const long long at = at_sh[rl];
      v[i] = at >= 0 ? *reinterpret_cast<const uint4*>(a.q.p + at + ch * 8) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t m = w[j] & 0x7fff7fffu;
        top = __vmaxu2(top, m & ~__vcmpgeu2(m, 0x7f807f80u));
      }
    }
    top = __reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xffffu));
    if ((tid & 31) == 0) top_sh[tid >> 5] = top;
    __syncthreads();
    top = max(max(top_sh[0], top_sh[1]), max(top_sh[2], top_sh[3])) >> 7;  // the largest's exponent
    const uint32_t up = top ? min(268u - top, 253u) : 127u;                // to 2^14 and more, as a float's exponent
    const float scale = __uint_as_float(up << 23);
    if (tid == 0) f.unit = __uint_as_float((254u - up) << 23);
    uint4* dst = g.packed + to * (kWcRows * CPR);
#pragma unroll
    for (int i = 0; i < N; ++i)
      dst[tile_off((i * 128 + tid) / CPR, (i * 128 + tid) % CPR) >> 4] = halves_of(v[i], scale);
    __syncthreads();
  }
}

static size_t up256w(size_t x) { return (x + 255) & ~(size_t)255; }
static long long weigh_tiles(int n_seqs, int total, int G) { return (long long)total * G / kWcRows + n_seqs + 1; }

size_t weigh_chunk_bytes(const entmaxkv_config& cfg, int n_seqs, int total) {
  const size_t segs = 2 * (size_t)kWcTurns * kWcMaxBlocks;
  return up256w((size_t)n_seqs * sizeof(WcSlot)) + up256w((size_t)(n_seqs + 1) * 8) +
         up256w((size_t)weigh_tiles(n_seqs, total, cfg.group) * (sizeof(WcRows) + 4)) + 256 + up256w(segs * 32) +
         (size_t)weigh_tiles(n_seqs, total, cfg.group) * cfg.num_kv_heads *
             (kWcRows * cfg.head_dim * 2 + sizeof(WcFacts)) +
         up256w(segs * kWcKeys * 4);
}

template <bool I8>
static cudaError_t weigh_chunk_d(const WcArgs& g, cudaStream_t st) {
  return g.a.c.D == 128 ? weigh_chunk_run<I8, 128>(g, st) : weigh_chunk_run<I8, 64>(g, st);
}

cudaError_t launch_weigh_chunk(const Q8WeighArgs& a, bool i8, void* ws, int sms, cudaStream_t st) {
  WcArgs g;
  g.a = a;
  g.blocks = min(sms, kWcMaxBlocks);
  const size_t tiles = (size_t)weigh_tiles(a.b.n_seqs, a.b.total, a.c.G), segs = 2 * (size_t)kWcTurns * kWcMaxBlocks;
  g.max_tiles = (int)tiles;
  char* p = static_cast<char*>(ws);
  g.slots = reinterpret_cast<WcSlot*>(p);
  p += up256w((size_t)a.b.n_seqs * sizeof(WcSlot));
  g.cum = reinterpret_cast<long long*>(p);
  p += up256w((size_t)(a.b.n_seqs + 1) * 8);
  g.rows = reinterpret_cast<WcRows*>(p);
  g.slot_of = reinterpret_cast<int*>(g.rows + tiles);
  p += up256w(tiles * (sizeof(WcRows) + 4));
  g.n_tiles = reinterpret_cast<int*>(p);
  p += 256;
  g.done = reinterpret_cast<int*>(p);
  p += up256w(segs * 32);
  g.part = reinterpret_cast<float*>(p);
  p += up256w(segs * kWcKeys * 4);
  g.packed = reinterpret_cast<uint4*>(p);
  p += tiles * a.c.Hkv * kWcRows * a.c.D * 2;
  g.facts = reinterpret_cast<WcFacts*>(p);
  cudaError_t e = launch_k(true, weigh_plan_kernel, dim3(1), dim3(1024), 0, st, g);
  const dim3 grid((unsigned)min(tiles, (size_t)65535), (unsigned)a.c.Hkv);
  if (e == cudaSuccess)
    e = a.c.D == 128 ? launch_k(true, weigh_pack_kernel<128>, grid, dim3(128), 0, st, g)
                     : launch_k(true, weigh_pack_kernel<64>, grid, dim3(128), 0, st, g);
  if (e != cudaSuccess) return e;
  return i8 ? weigh_chunk_d<true>(g, st) : weigh_chunk_d<false>(g, st);
}

}  // namespace ekv
