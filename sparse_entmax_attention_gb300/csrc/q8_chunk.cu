// q8_chunk.cu -- the item list, the joining kernel and the launches of the
// chunk attention (q8_chunk.cuh).
#include "q8_chunk.cuh"

namespace ekv {

template <>
cudaError_t chunk_run<true, 128, false>(const ChunkArgs& g, cudaStream_t st);
template <>
cudaError_t chunk_run<true, 128, true>(const ChunkArgs& g, cudaStream_t st);
template <>
cudaError_t chunk_run<true, 64, false>(const ChunkArgs& g, cudaStream_t st);
template <>
cudaError_t chunk_run<true, 64, true>(const ChunkArgs& g, cudaStream_t st);
template <>
cudaError_t chunk_run<false, 128, false>(const ChunkArgs& g, cudaStream_t st);
template <>
cudaError_t chunk_run<false, 128, true>(const ChunkArgs& g, cudaStream_t st);
template <>
cudaError_t chunk_run<false, 64, false>(const ChunkArgs& g, cudaStream_t st);
template <>
cudaError_t chunk_run<false, 64, true>(const ChunkArgs& g, cudaStream_t st);

// One block lists the items and the line: slots 1024 at a time, then the
// round's items, a thread each.
__global__ void __launch_bounds__(1024) chunk_plan_kernel(ChunkArgs g) {
  pdl_enter();
  __shared__ int sh_scan[32];
  __shared__ int end_sh[1024];
  const Q8AttendArgs& a = g.a;
  const int tid = threadIdx.x, per = kChunkKeys / a.c.P;
  __shared__ int none_sh;
  if (tid == 0) none_sh = 0;
  int items = 0, tiles = 0;
  for (int b0 = 0; b0 < a.b.n_seqs; b0 += 1024) {
    const int b = b0 + tid;
    int nrt = 0;
    if (b < a.b.n_seqs) {
      const Q8Slot s = q8_slot(a.c, a.b, b, a.c.status);
      nrt = (int)(((long long)s.count * a.c.G + kChunkRows - 1) / kChunkRows);
    }
    int total;
    const int at = block_exclusive_scan(nrt, sh_scan, total);
    end_sh[tid] = at + nrt;
    __syncthreads();
    for (int j0 = 0; j0 < total; j0 += 1024) {
      const int j = j0 + tid;
      int T = 0, lo = 0;
      if (j < total) {
        int hi = 1023;
        while (lo < hi) {
          const int m = (lo + hi) >> 1;
          if (end_sh[m] > j) hi = m;
          else lo = m + 1;
        }
        const int rt = j - (lo ? end_sh[lo - 1] : 0);
        const Q8Slot s = q8_slot(a.c, a.b, b0 + lo, nullptr);
        const Q8Span v = chunk_span(a, s, b0 + lo, rt);
        T = (v.T + per - 1) / per;
        if (items + j < g.max_items) {
          g.items[items + j] = ChunkItem{b0 + lo, rt, T, v.T, s.seq, s.L, s.start, s.count, v.pre, v.npre, v.wfirst, v.npages};
          if (T == 0) g.empty[atomicAdd(&none_sh, 1)] = items + j;  // (any order will do)
        } else {  // rows that several slots claim: the items past the list get no place on the line
          T = 0;
          raise_flag(a.c.status, ENTMAXKV_DEV_BAD_BATCH);
        }
      }
      int all;
      const int before = block_exclusive_scan(T ? T + kChunkItem : 0, sh_scan, all);
      if (j < total && items + j < g.max_items) g.cum[items + j] = tiles + before;
      tiles += all;
    }
    items = min(items + total, g.max_items);  // (rows claimed over and over: the sum may pass 31 bits)
    __syncthreads();
  }
  if (tid == 0) {
    g.n_items[0] = items;
    g.n_items[1] = none_sh;
    g.cum[items] = tiles;
  }
}

// Joins items that several blocks hold: at each block that begins inside an
// item it shares with the block before it alone or first. Eight blocks a cut,
// 32 rows each, a warp a row; the first eight answer rows that see no key.
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(ChunkArgs g) {
  pdl_enter();
  const Q8AttendArgs& a = g.a;
  const int c = blockIdx.x >> 3, part = blockIdx.x & 7, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.c.G, Hkv = a.c.Hkv;
  constexpr int V = D / 32;
  if (c == 0) {
    const long long n = (long long)g.n_items[1] * Hkv;
    for (long long i = part; i < n; i += 8) {
      const ChunkItem it = g.items[g.empty[i / Hkv]];
      for (int row = warp; row < kChunkRows; row += 8) {
        const int rho = it.rt * kChunkRows + row;
        if (rho >= it.count * G) break;
        const int head = (int)(i % Hkv) * G + rho % G;
        const long long tok = it.start + rho / G;
        const int to = a.lam ? head >> 1 : head;  // (a pair's rows write the same zeros)
        for (int k = lane; k < D; k += 32) a.out.p[tok * a.out.ts + (long long)to * a.out.hs + k] = __float2bfloat16_rn(0.0f);
        if (a.tau && lane == 0) a.tau[tok * Hkv * G + head] = CUDART_NAN_F;
      }
    }
    return;
  }
  const int2 cut = g.cuts[c];
  if (cut.x < 0) return;
  const ChunkItem it = g.items[cut.x];
  const int cum = g.cum[cut.x], S = g.cum[g.n_items[0]];
  const long long W = (long long)S * Hkv, nb = max(1LL, min(W, (long long)g.blocks));
  const long long A = (long long)cut.y * S + cum + kChunkItem;
  const int c0 = (int)(((A + 1) * nb - 1) / W), n = (int)(((A + it.T) * nb - 1) / W) - c0 + 1;
  if (c0 != c - 1) return;  // joined at an earlier cut
  const int last0 = W * c0 / nb >= A - kChunkItem ? 0 : 1;  // the first block's piece: its first or its last
  auto row_sum = [&](int row, float& M, float& l, float (&o)[V]) {
    auto piece = [&](int i) -> size_t { return (size_t)(2 * (c0 + i) + (i ? 0 : last0)) * kChunkRows + row; };
    M = -CUDART_INF_F;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.0f;
    for (int i0 = 0; i0 < n; i0 += 32) {  // 32 pieces' maxima and sums at once, one a lane
      float2 ml = make_float2(-CUDART_INF_F, 0.0f);
      if (i0 + lane < n) ml = g.part_ml[piece(i0 + lane)];
      const float m = fmaxf(M, warp_max(ml.x));
      const float old = M > -CUDART_INF_F ? ex2f(M - m) : 0.0f, f = ml.x > -CUDART_INF_F ? ex2f(ml.x - m) : 0.0f;
      l = l * old + warp_sum(f * ml.y);
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] *= old;
      M = m;
      const int m32 = min(32, n - i0);
#pragma unroll 4
      for (int i = 0; i < m32; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i);
        const float* p = g.part_o + piece(i0 + i) * D + lane;
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = fmaf(fi, p[32 * k], o[k]);
      }
    }
  };
  if (a.lam) {  // a warp a pair
    for (int row = 32 * part + 2 * warp; row < 32 * part + 32; row += 16) {
      const int rho = it.rt * kChunkRows + row;
      if (rho >= it.count * G) break;
      float M[2], l[2], o[V], o1[V], sum2 = 0.0f;
      row_sum(row, M[0], l[0], o);
      row_sum(row + 1, M[1], l[1], o1);
      const int head = cut.y * G + rho % G;
      const long long tok = it.start + rho / G;
      const float i0 = att_inv(l[0]), i1 = att_inv(l[1]) * a.lam[tok * a.lam_ts + (head >> 1)];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        o[i] = diff_of(o[i], i0, o1[i], i1);
        sum2 = fmaf(o[i], o[i], sum2);
      }
      if (a.gain) {
        const float f = diff_norm_warp(a, o, sum2);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] *= f * a.gain[32 * i + lane];
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        a.out.p[tok * a.out.ts + (long long)(head >> 1) * a.out.hs + 32 * i + lane] = __float2bfloat16_rn(o[i]);
      if (a.tau && lane < 2) a.tau[tok * Hkv * G + head + lane] = lane ? att_lse(M[1], l[1]) : att_lse(M[0], l[0]);
    }
    return;
  }
#pragma unroll 2
  for (int row = 32 * part + warp; row < 32 * part + 32; row += 8) {
    const int rho = it.rt * kChunkRows + row;
    if (rho >= it.count * G) break;
    float M, l, o[V];
    row_sum(row, M, l, o);
    const int head = cut.y * G + rho % G;
    const long long tok = it.start + rho / G;
    const float inv = att_inv(l);
#pragma unroll
    for (int i = 0; i < V; ++i)
      a.out.p[tok * a.out.ts + (long long)head * a.out.hs + 32 * i + lane] = __float2bfloat16_rn(o[i] * inv);
    if (a.tau && lane == 0) a.tau[tok * Hkv * G + head] = att_lse(M, l);
  }
}

static long long chunk_items(int n_seqs, int total, int G) {
  return (long long)total * G / kChunkRows + n_seqs + 1;
}
// A KV head's line is counted in 32 bits.
bool chunk_counts_fit(const entmaxkv_config& cfg, int n_seqs, int total) {
  const long long keys = (long long)cfg.max_pages_per_seq * cfg.page_size;
  return chunk_items(n_seqs, total, cfg.group) <= 0x7fffffffLL / ((keys + kChunkKeys - 1) / kChunkKeys + kChunkItem);
}

static size_t up256c(size_t x) { return (x + 255) & ~(size_t)255; }

size_t attend_chunk_bytes(const entmaxkv_config& cfg, int n_seqs, int total) {
  const size_t items = (size_t)chunk_items(n_seqs, total, cfg.group);
  return up256c(items * sizeof(ChunkItem)) + up256c((items + 1) * 4) + 256 + up256c(items * 4) +
         up256c((size_t)kChunkMaxBlocks * 8) +
         up256c((size_t)kChunkMaxBlocks * 2 * kChunkRows * cfg.head_dim * 4) +
         up256c((size_t)kChunkMaxBlocks * 2 * kChunkRows * 8);
}

template <bool I8>
static cudaError_t chunk_d(ChunkArgs& g, cudaStream_t st) {
  if (g.a.lam) return g.a.c.D == 128 ? chunk_run<I8, 128, true>(g, st) : chunk_run<I8, 64, true>(g, st);
  return g.a.c.D == 128 ? chunk_run<I8, 128, false>(g, st) : chunk_run<I8, 64, false>(g, st);
}

cudaError_t launch_attend_chunk(const Q8AttendArgs& a, bool i8, void* ws, int sms, cudaStream_t st) {
  ChunkArgs g;
  g.a = a;
  const size_t items = (size_t)chunk_items(a.b.n_seqs, a.b.total, a.c.G);
  g.max_items = (int)items;
  g.blocks = min(sms, kChunkMaxBlocks);
  char* p = static_cast<char*>(ws);
  g.items = reinterpret_cast<ChunkItem*>(p);
  p += up256c(items * sizeof(ChunkItem));
  g.cum = reinterpret_cast<int*>(p);
  p += up256c((items + 1) * 4);
  g.n_items = reinterpret_cast<int*>(p);
  p += 256;
  g.empty = reinterpret_cast<int*>(p);
  p += up256c(items * 4);
  g.cuts = reinterpret_cast<int2*>(p);
  p += up256c((size_t)kChunkMaxBlocks * 8);
  g.part_o = reinterpret_cast<float*>(p);
  p += up256c((size_t)kChunkMaxBlocks * 2 * kChunkRows * a.c.D * 4);
  g.part_ml = reinterpret_cast<float2*>(p);
  cudaError_t e = launch_k(false, chunk_plan_kernel, dim3(1), dim3(1024), 0, st, g);
  if (e == cudaSuccess) e = i8 ? chunk_d<true>(g, st) : chunk_d<false>(g, st);
  if (e != cudaSuccess) return e;
  return a.c.D == 128 ? launch_k(true, chunk_join_kernel<128>, dim3(8 * g.blocks), dim3(256), 0, st, g)
                      : launch_k(true, chunk_join_kernel<64>, dim3(8 * g.blocks), dim3(256), 0, st, g);
}

}  // namespace ekv
