// q8_chunk.cu -- the item list, the joining kernel and the launches of the
// chunk attention (q8_chunk.cuh).
#include "q8_chunk.cuh"

namespace ekv {

template <>
cudaError_t chunk_run<true, 128>(const ChunkArgs& g, cudaStream_t st);
template <>
cudaError_t chunk_run<true, 64>(const ChunkArgs& g, cudaStream_t st);
template <>
cudaError_t chunk_run<false, 128>(const ChunkArgs& g, cudaStream_t st);
template <>
cudaError_t chunk_run<false, 64>(const ChunkArgs& g, cudaStream_t st);

// One block lists the items and the line: slots 1024 at a time, then the
// round's items, a thread each.
__global__ void __launch_bounds__(1024) chunk_plan_kernel(ChunkArgs g) {
  pdl_enter();
  __shared__ int sh_scan[32];
  __shared__ int end_sh[1024];
  const Q8AttendArgs& a = g.a;
  const int tid = threadIdx.x, per = kChunkKeys / a.c.P;
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
        T = (chunk_span(a, s, b0 + lo, rt).T + per - 1) / per;
        if (items + j < g.max_items) g.items[items + j] = ChunkItem{b0 + lo, rt};
      }
      int all;
      const int before = block_exclusive_scan(T, sh_scan, all);
      if (j < total && items + j < g.max_items) g.cum[items + j] = tiles + before;
      tiles += all;
    }
    items += total;
    __syncthreads();
  }
  if (tid == 0) {
    items = min(items, g.max_items);  // (slots whose rows overlap can claim more: those are not answered)
    *g.n_items = items;
    g.cum[items] = tiles;
  }
}

// Joins items that several blocks hold and answers rows that see no key.
// Block (item · KV head, 8 rows): a warp a row.
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(ChunkArgs g) {
  pdl_enter();
  const Q8AttendArgs& a = g.a;
  const int item = blockIdx.x / a.c.Hkv, kvh = blockIdx.x % a.c.Hkv, n_items = *g.n_items;
  if (item >= n_items) return;
  const ChunkItem it = g.items[item];
  const Q8Slot s = q8_slot(a.c, a.b, it.slot, nullptr);
  const int S = g.cum[n_items], G = a.c.G;
  const long long W = (long long)S * a.c.Hkv, nb = max(1LL, min(W, (long long)g.blocks));
  const int T = g.cum[item + 1] - g.cum[item];
  const long long A = (long long)kvh * S + g.cum[item];
  long long c0 = 0, c1 = -1;
  if (T > 0) {
    c0 = ((A + 1) * nb - 1) / W;
    c1 = ((A + T) * nb - 1) / W;
    if (c0 == c1) return;  // finished by that block
  }
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5), rho = it.rt * kChunkRows + row;
  if (rho >= s.count * G) return;
  auto piece = [&](long long c) -> size_t {
    return ((size_t)(2 * c + (W * c / nb >= A ? 0 : 1))) * kChunkRows + row;
  };
  float M = -CUDART_INF_F, l = 0.0f;
  constexpr int V = D / 32;
  float o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.0f;
  for (long long c = c0; c <= c1; ++c) M = fmaxf(M, g.part_ml[piece(c)].x);
#pragma unroll 2
  for (long long c = c0; c <= c1; ++c) {
    const float2 ml = g.part_ml[piece(c)];
    const float f = ml.x > -CUDART_INF_F ? ex2f(ml.x - M) : 0.0f;
    l = fmaf(f, ml.y, l);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = fmaf(f, g.part_o[piece(c) * D + 32 * i + lane], o[i]);
  }
  const int head = kvh * G + rho % G;
  const long long tok = s.start + rho / G;
  const float inv = att_inv(l);
#pragma unroll
  for (int i = 0; i < V; ++i)
    a.out.p[tok * a.out.ts + (long long)head * a.out.hs + 32 * i + lane] = __float2bfloat16_rn(o[i] * inv);
  if (a.tau && lane == 0) a.tau[tok * a.c.Hkv * G + head] = att_lse(M, l);
}

static size_t up256c(size_t x) { return (x + 255) & ~(size_t)255; }
static long long chunk_items(int n_seqs, int total, int G) {
  return (long long)total * G / kChunkRows + n_seqs + 1;
}

size_t attend_chunk_bytes(const entmaxkv_config& cfg, int n_seqs, int total) {
  const size_t items = (size_t)chunk_items(n_seqs, total, cfg.group);
  return up256c(items * sizeof(ChunkItem)) + up256c((items + 1) * 4) + 256 +
         up256c((size_t)kChunkMaxBlocks * 2 * kChunkRows * cfg.head_dim * 4) +
         up256c((size_t)kChunkMaxBlocks * 2 * kChunkRows * 8);
}

template <bool I8>
static cudaError_t chunk_d(ChunkArgs& g, cudaStream_t st) {
  return g.a.c.D == 128 ? chunk_run<I8, 128>(g, st) : chunk_run<I8, 64>(g, st);
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
  g.part_o = reinterpret_cast<float*>(p);
  p += up256c((size_t)kChunkMaxBlocks * 2 * kChunkRows * a.c.D * 4);
  g.part_ml = reinterpret_cast<float2*>(p);
  cudaError_t e = launch_k(false, chunk_plan_kernel, dim3(1), dim3(1024), 0, st, g);
  if (e == cudaSuccess) e = i8 ? chunk_d<true>(g, st) : chunk_d<false>(g, st);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(g.max_items * a.c.Hkv), kChunkRows / 8);
  return a.c.D == 128 ? launch_k(false, chunk_join_kernel<128>, grid, dim3(256), 0, st, g)
                      : launch_k(false, chunk_join_kernel<64>, grid, dim3(256), 0, st, g);
}

}  // namespace ekv
