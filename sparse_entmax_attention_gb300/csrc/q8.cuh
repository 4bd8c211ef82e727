// q8.cuh -- what the kernels of the 8-bit paged cache share: the batch's
// slots, the code types and the argument blocks. Internal.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace ekv {

// The cache and the batch, as every kernel takes them.
struct Q8Cache {
  int Hkv, G, D, P, maxp, nphys, max_seqs;
  uint8_t* k_pool;
  uint8_t* v_pool;
  float* k_scale;
  float* v_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  uint32_t* status;
};
struct Q8Batch {
  const int32_t* seq_ids;
  const int32_t* start;
  const int32_t* count;
  int n_seqs, total, max_count;
};
struct Q8Rows {
  __nv_bfloat16* p;
  long long ts, hs;  // strides in elements: token, head
};

// Slot b of the batch: its sequence row, length, first row and row count;
// count 0 when it is idle or refused (flagged on st, which may be null).
struct Q8Slot {
  int seq, L, start, count;
};
__device__ __forceinline__ Q8Slot q8_slot(const Q8Cache& c, const Q8Batch& b, int i, uint32_t* st) {
  Q8Slot s{-1, 0, 0, 0};
  const int n = b.count[i], start = b.start[i], seq = b.seq_ids ? b.seq_ids[i] : i;  // (one round trip)
  if (n == 0) return s;
  s.start = start;
  if (seq < 0 || seq >= c.max_seqs) {
    raise_flag(st, ENTMAXKV_DEV_BAD_SEQ_ID);
    return s;
  }
  s.seq = seq;
  s.L = seq_len_clamped(c.seq_lens, s.seq, c.maxp, c.P, st);
  if (n < 0 || n > b.max_count || n > s.L || s.start < 0 || (long long)s.start + n > b.total) {
    raise_flag(st, ENTMAXKV_DEV_BAD_BATCH);
    return s;
  }
  s.count = n;
  return s;
}

// Four e4m3 codes -> halves (exact): bytes 0 and 1 to x, 2 and 3 to y.
__device__ __forceinline__ void e4m3x4_half(uint32_t w, uint32_t& x, uint32_t& y) {
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n cvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
      : "=r"(x), "=r"(y)
      : "r"(w));
}

// Four codes of a word as halves, exact: even holds bytes 0 and 2, odd bytes 1
// and 3 (SPLIT) or lo bytes 0 and 1, hi bytes 2 and 3. Whole numbers: the byte
// with its sign bit flipped is u = v + 128, 0x6400 | u is the half 1024 + u,
// and 1024 + u - 1152 = v.
template <bool I8, bool SPLIT>
__device__ __forceinline__ void codes_half(uint32_t w, uint32_t& x, uint32_t& y) {
  if constexpr (I8) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, SPLIT ? 0x4240 : 0x4140);
    const uint32_t b = __byte_perm(u, 0x64646464u, SPLIT ? 0x4341 : 0x4342);
    const __half2 off = __float2half2_rn(-1152.0f);
    const __half2 ha = __hadd2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 hb = __hadd2(*reinterpret_cast<const __half2*>(&b), off);
    x = *reinterpret_cast<const uint32_t*>(&ha);
    y = *reinterpret_cast<const uint32_t*>(&hb);
  } else {
    e4m3x4_half(SPLIT ? __byte_perm(w, 0u, 0x3120) : w, x, y);
  }
}

// One code as a float (exact).
template <bool I8>
__device__ __forceinline__ float code_f(uint32_t byte) {
  if constexpr (I8) return (float)(int)(int8_t)(byte & 0xffu);
  uint32_t x, y;
  e4m3x4_half(byte & 0xffu, x, y);
  return __low2float(*reinterpret_cast<const __half2*>(&x));
}

// D = A·B + D for one m16n8k16 tile, fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8×8 tile of halves held as mma fragments.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float ex2f(float x) {  // 2^x, relative error about 2^-22
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// How the scores are formed (defaults already filled in).
struct Q8Score {
  float scale, cap, inv_cap;
  int window;
  const float* slopes;
  const int32_t* prefix;
  const int32_t* first_key;
};

constexpr float kLog2e = 1.4426950408889634f;

// cap·tanh(s/cap) as cap·(1 − 2/(1 + e^{2s/cap})): absolute error about
// cap·2^-22, which is what a score's error costs its weight.
__device__ __forceinline__ float soft_cap(float s, float cap, float inv_cap) {
  const float e = ex2f(2.0f * kLog2e * inv_cap * s);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return cap * fmaf(-2.0f, r, 1.0f);
}

// Visible keys of a slot's rows: pages [0, npre) hold the prefix and pages
// [wfirst, npages) what window and documents leave; T pages in all, the t-th
// being page(t).
struct Q8Span {
  int pre, npre, wfirst, npages, T;
  __device__ __forceinline__ int page(int t) const { return t < npre ? t : t - npre + wfirst; }
};
// The span of rows [r0, r0 + n) of slot b.
__device__ __forceinline__ Q8Span q8_span(const Q8Cache& c, const Q8Score& sc, const Q8Slot& s, int b, int r0, int n) {
  Q8Span v;
  const int x0 = s.L - s.count + r0, end = x0 + n;  // positions [x0, end)
  v.pre = sc.prefix ? min(max(sc.prefix[b], 0), s.L) : 0;
  int lo = sc.window > 0 ? max(0, x0 - sc.window + 1) : 0;
  if (sc.first_key) {
    int fk = 0x7fffffff;
#pragma unroll 8
    for (int i = 0; i < n; ++i) fk = min(fk, sc.first_key[s.start + r0 + i]);
    lo = max(lo, fk);
  }
  v.npages = max((end + c.P - 1) / c.P, (v.pre + c.P - 1) / c.P);
  v.wfirst = lo >= end ? v.npages : lo / c.P;
  v.npre = min((v.pre + c.P - 1) / c.P, v.wfirst);
  // keys behind `end` belong to the prefix alone
  v.T = v.npre + v.npages - v.wfirst;
  return v;
}

struct Q8AttendArgs {
  Q8Cache c;
  Q8Batch b;
  Q8Score sc;
  Q8Rows q, out;
  float* tau;
  // differential attention (lam not null): out has a head a pair of query heads, their difference
  const float* lam;   // factor of pair i in row t: lam[t·lam_ts + i]
  long long lam_ts;
  const float* gain;  // [D] of the difference's norm over its head, or null: none
  float eps;
  // workspace
  long long* cum;   // [n_seqs + 1] tiles before each slot
  void* slots;      // [n_seqs] what the streaming kernel made of each slot
  float* part_o;    // [blocks][2][rows][D]
  float* part_ml;   // [blocks][2][rows][2] running max (base 2) and sum
  int blocks;
};

// o0·i0 − o1·i1, both products rounded: equal maps with a factor of 1 cancel to 0.
__device__ __forceinline__ float diff_of(float o0, float i0, float o1, float i1) {
  return __fsub_rn(__fmul_rn(o0, i0), __fmul_rn(o1, i1));
}
// What a pair's difference y is multiplied by, dim by dim gain's: 1/√(mean y² + ε), from Σ (y·down)². down is 1, or
// where that sum passes fp32 (values of 2^60 and more) 2^-70: then it lies between 2^-12 and 2^123.
constexpr float kDiffDown = 0x1p-70f;
__device__ __forceinline__ bool diff_past(float sum2) { return sum2 > 0x1.fffffep127f; }
__device__ __forceinline__ float diff_norm(const Q8AttendArgs& a, float sum2, float down = 1.0f) {
  return down * rsqrtf(fmaf(sum2, 1.0f / (float)a.c.D, a.eps * down * down));
}

struct Q8WeighArgs {
  Q8Cache c;
  Q8Batch b;
  Q8Score sc;
  Q8Rows q;
  const float* tau;      // [total][Hq]
  const float* coef;     // [total][Hq], or null: 1
  const int32_t* fresh;  // [n_seqs] last keys whose weight begins at 0, or null: the batch's rows
  float* w;              // [num_phys_pages][Hkv][page_size]
  float decay, a1, beta; // a1 = α − 1 (0: softmax), beta = 1/a1
};

cudaError_t launch_plan(const entmaxkv_config& cfg, int32_t* block_table, const int32_t* seq_lens, uint32_t* status,
                        const int32_t* seq_ids, const int32_t* n_new, int n_seqs, int total, int max_count,
                        const int32_t* free_pages, const int32_t* free_count, int32_t* free_count_out,
                        int32_t* lens_out, int32_t* start, int32_t* count, int32_t* positions, int64_t* slots,
                        cudaStream_t st);
cudaError_t launch_release(const entmaxkv_config& cfg, const int32_t* block_table, int32_t* seq_lens, uint32_t* status,
                           const int32_t* seq_ids, int n_seqs, int32_t* free_pages, int32_t* free_count,
                           cudaStream_t st);
cudaError_t launch_append_q8(const Q8Cache& c, const Q8Batch& b, const Q8Rows& k, const Q8Rows& v, bool i8, int sms,
                             cudaStream_t st);
cudaError_t launch_read_q8(const Q8Cache& c, const Q8Batch& b, const int32_t* first, const Q8Rows& k, const Q8Rows& v,
                           bool i8, int sms, cudaStream_t st);
size_t attend_softmax_bytes(const entmaxkv_config& cfg, int n_seqs);
cudaError_t launch_attend_softmax(Q8AttendArgs a, bool i8, void* ws, int sms, cudaStream_t st);
// Rows (tokens times the group) of a batch's largest slot up to which the
// streaming kernel answers the batch, 16 rows at a time; with more, 128-row product
// tiles do. Measured, streaming against products, batches of equal slots, int8, 4 KV
// heads: 24 sequences of 6000 tokens at d = 128 46/99 us at 16 rows, 77/104 at 32,
// 108/105 at 48, 137/105 at 64; 4 of 30000 (pages of 16) 46/95, 67/103, 94/104,
// 117/107; 24 of 6000 at d = 64 36/62, 50/67, 68/66, 86/66. A batch of unequal slots
// is not split: 24 decodes of 4k-29k tokens (8 KV heads, d = 128) take 142 us and a
// chunk of 1000 behind 8000 151 us, both in one call 576 us.
constexpr int kStreamRows = 48;
bool chunk_counts_fit(const entmaxkv_config& cfg, int n_seqs, int total);
size_t attend_chunk_bytes(const entmaxkv_config& cfg, int n_seqs, int total);
cudaError_t launch_attend_chunk(const Q8AttendArgs& a, bool i8, void* ws, int sms, cudaStream_t st);
size_t attend_entmax_bytes(const entmaxkv_config& cfg, int n_seqs);
cudaError_t launch_attend_entmax(const entmaxkv_config& cfg, Q8AttendArgs a, bool i8, float alpha, void* ws, int sms,
                                 cudaStream_t st);
// Rows of a batch's largest slot up to which the streaming kernel weighs keys; with
// more, 128-row product tiles do. 32 is what the streaming kernel's largest variant
// holds (four tiles of 8 rows in registers), not where the two cross: it is still ahead
// there. Measured, streaming against products, batches of equal slots, int8, 8 KV heads:
// 24 sequences of 6000 tokens at d = 128 43/90 us at 16 rows, 70/92 at 32; 4 of 30000
// 37/75, 61/78; one of 32768 17/31, 23/33; 24 of 6000 at d = 64 31/74, 55/80.
constexpr int kWeighRows = 32;
size_t weigh_chunk_bytes(const entmaxkv_config& cfg, int n_seqs, int total);
cudaError_t launch_weigh_chunk(const Q8WeighArgs& a, bool i8, void* ws, int sms, cudaStream_t st);
cudaError_t launch_weigh_stream(const Q8WeighArgs& a, bool i8, int sms, cudaStream_t st);
size_t evict_bytes(const entmaxkv_config& cfg, int n, int keep);
cudaError_t launch_evict(const Q8Cache& c, const int32_t* seq_ids, const int32_t* count, int n, int keep, int above, int sinks, int recent,
                         const float* w, float* w_out, int32_t* lens_out, int32_t* free_pages,
                         const int32_t* free_count, int32_t* count_out, bool i8, void* ws, int sms, cudaStream_t st);
// A pool as (dim, KV head · token, page) of bytes, in boxes of one slab.
cudaError_t make_q8_map(CUtensorMap* map, const void* pool, int nphys, int Hkv, int P, int D);

}  // namespace ekv
