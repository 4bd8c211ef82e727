// q8_tiles.cuh -- pieces of the kernels that stream 8-bit pages through shared
// memory: the slab layout, K and V fragments, query fragments. Internal.
#pragma once

#include "q8.cuh"

namespace ekv {

// A slab of P rows of D codes arrives by a swizzled tensor copy (128- or
// 64-byte swizzle for D = 128 or 64): byte offset of 16-byte chunk ch of row t.
// The copies below and ldmatrix then touch eight different 16-byte banks a
// phase.
template <int D>
__device__ __forceinline__ uint32_t slab_off(int t, int ch) {
  if constexpr (D == 128) return (uint32_t)(t * 128 + ((ch ^ (t & 7)) << 4));
  return (uint32_t)(t * 64 + ((ch ^ ((t >> 1) & 3)) << 4));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
  return r;
}

// A query row as mma B fragments in halves: lane (n = lane/4, c = lane%4) holds
// dims (D/4)·c + 4ks .. +3 of row n, the order in which a lane's K bytes lie.
// A power of two brings the row's largest value into [2^13, 2^14), so bf16
// values down to 2^-27 of it are exact as halves; inv is that power's inverse. A
// row that holds an infinity or a NaN becomes all NaN, and so do its scores (an
// infinity alone could make all of them −∞, which is a masked key's).
// p = null: a row of zeros.
template <int D>
__device__ __forceinline__ void q_load(const __nv_bfloat16* p, int lane, uint4 (&w)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    w[i] = p ? *reinterpret_cast<const uint4*>(p + (D / 4) * (lane & 3) + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
}
template <int D>
__device__ __forceinline__ void q_half_frag(const uint4 (&w)[D / 32], uint32_t (&b)[D / 16][2], float& inv) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    m = __vmaxu2(__vmaxu2(m, w[i].x & 0x7fff7fffu), w[i].y & 0x7fff7fffu);
    m = __vmaxu2(__vmaxu2(m, w[i].z & 0x7fff7fffu), w[i].w & 0x7fff7fffu);
  }
  m = max(m & 0xffffu, m >> 16);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  int e = (int)(m >> 7) - 127;
  e = max(e, -100);
  const float f = m >= 0x7f80u ? CUDART_NAN_F : __uint_as_float((uint32_t)(13 - e + 127) << 23);
  inv = __uint_as_float((uint32_t)(e - 13 + 127) << 23);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 x = __floats2half2_rn(bf_lo(u[j]) * f, bf_hi(u[j]) * f);
      b[2 * i + (j >> 1)][j & 1] = *reinterpret_cast<const uint32_t*>(&x);
    }
  }
}

// acc[nt] = codes of 16 tokens (rows from token t16) · query rows 8nt..8nt+7:
// lane l holds tokens l/4 and l/4 + 8 of rows 2(l%4), 2(l%4) + 1.
template <bool I8, int D, int NT>
__device__ __forceinline__ void k_dot(uint32_t slab, int t16, int lane, const uint32_t (&bq)[NT][D / 16][2],
                                      float (&acc)[NT][4]) {
  const int r = lane >> 2, c = lane & 3;
  constexpr int CH = D / 64;  // 16-byte chunks a lane holds of a row
  uint4 x[2][CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    x[0][j] = lds128(slab + slab_off<D>(t16 + r, CH * c + j));
    x[1][j] = lds128(slab + slab_off<D>(t16 + r + 8, CH * c + j));
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const int j = ks >> 2, w = ks & 3;
    const uint32_t w0 = w == 0 ? x[0][j].x : w == 1 ? x[0][j].y : w == 2 ? x[0][j].z : x[0][j].w;
    const uint32_t w1 = w == 0 ? x[1][j].x : w == 1 ? x[1][j].y : w == 2 ? x[1][j].z : x[1][j].w;
    uint32_t a0, a1, a2, a3;
    codes_half<I8, false>(w0, a0, a2);
    codes_half<I8, false>(w1, a1, a3);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], a0, a1, a2, a3, bq[nt][ks][0], bq[nt][ks][1]);
  }
}

// tmp[mt][nt] += V^T of 16 tokens (from t16) · p: b[nt] are p's B fragments.
// Lane l's sums are of dims 16mt + 2(l/4) (elements 0, 1) and the next one
// (elements 2, 3), for rows 2(l%4) and 2(l%4) + 1.
template <bool I8, int D, int NT>
__device__ __forceinline__ void v_dot(uint32_t slab, int t16, int lane, const uint32_t (&b)[NT][2],
                                      float (&tmp)[D / 16][NT][4]) {
  const int t = t16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
  for (int mt = 0; mt < D / 16; mt += 2) {
    uint32_t w0, w1, w2, w3;
    ldsm_x4_trans(w0, w1, w2, w3, slab + slab_off<D>(t, mt + (lane >> 4)));
    uint32_t a0, a1, a2, a3;
    codes_half<I8, true>(w0, a0, a1);
    codes_half<I8, true>(w1, a2, a3);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mma_f16(tmp[mt][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
    codes_half<I8, true>(w2, a0, a1);
    codes_half<I8, true>(w3, a2, a3);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mma_f16(tmp[mt + 1][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
  }
}

// tanh(y) = y·T(y²): T interpolates tanh(√z)/√z at the Chebyshev points of
// [0, 1/4] (degree 3, relative error below 7e-7 in fp32 for |y| ≤ 1/2) and of
// [0, 1] (degree 6, below 1.5e-7), both against tanh in 64 bits at 20001 points.
struct TanhPoly {
  float near[4], far[7];
};
__device__ __forceinline__ constexpr TanhPoly tanh_poly() {
  return TanhPoly{{0.99999946f, -0.33326283f, 0.1318994f, -0.04439274f},
                  {0.99999994f, -0.33332828f, 0.13325076f, -0.053451646f, 0.020279707f, -0.0061943247f, 0.0010380251f}};
}
// Maxima in which a NaN stays.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Weights are 2^{t − M + kLift}; M moves when a t passes it by more than kSlack.
constexpr float kLift = 8.0f, kSlack = 6.0f;
constexpr int kNoKey = 0x40000000;  // first key of a place without a page: beyond every key

// What a lane knows of the two rows of an mma column pair. Scores come in
// units of 1/unit: unit = log2(e) for a softmax in base 2, α − 1 for entmax.
struct Q8Row {
  float cs;     // of the fp32 dot product (times the page's K scale): the score's, or with a cap score/cap's, units
  float slope;  // times unit
  int pos, lo;  // position, first key seen
};
__device__ __forceinline__ float q8_row_scale(float q_inv, const Q8Score& sc, float unit) {
  return q_inv * sc.scale * (sc.cap > 0.0f ? sc.inv_cap : unit);
}

// Scores of N keys for one row: dot[i] is of key j0 + 8·i; add is added to
// each. NaN-free for finite codes.
template <int N>
__device__ __forceinline__ void q8_scores(const float (&dot)[N], float (&out)[N], const Q8Row& r, float ks, int j0,
                                          const Q8Score& sc, float unit, float add) {
  const float k = r.cs * ks;
  if (sc.cap > 0.0f) {
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      out[i] = dot[i] * k;
      big = fmaxf(big, fabsf(out[i]));
    }
    constexpr TanhPoly poly = tanh_poly();
    const float c = sc.cap * unit;
    if (__all_sync(0xffffffffu, big <= 0.5f)) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float z = out[i] * out[i];
        const float t = fmaf(fmaf(fmaf(poly.near[3], z, poly.near[2]), z, poly.near[1]), z, poly.near[0]);
        out[i] = fmaf(t * out[i], c, add);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = fmaf(soft_cap(out[i], 1.0f, 1.0f), c, add);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = fmaf(dot[i], k, add);
  }
  if (sc.slopes) {
    const float d = (float)(r.pos - j0);
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = fmaf(fabsf(d - 8.0f * i), -r.slope, out[i]);
  }
}
__device__ __forceinline__ bool q8_sees(const Q8Row& r, int j, int pre) { return (j >= r.lo && j <= r.pos) || j < pre; }

// Wait for a phase of an mbarrier for at most a second.
__device__ __forceinline__ bool mbar_wait_second(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %globaltimer;\n" : "=l"(t0));
  do {
    if (mbar_try_wait(bar, parity)) return true;
    asm volatile("mov.u64 %0, %globaltimer;\n" : "=l"(t));
  } while (t - t0 < 1000000000ull);
  return false;
}

// One row's answer from its sums.
__device__ __forceinline__ float att_inv(float l) { return l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : CUDART_NAN_F); }
__device__ __forceinline__ float att_lse(float m, float l) {
  return l != 0.0f ? (m + log2f(l)) * 0.6931471805599453f : CUDART_NAN_F;
}

// n / d for n ≥ 0, d > 0: in 32 bits where both fit (the 64-bit division is a
// long subroutine, and code that runs once costs its instructions' fetch).
__device__ __forceinline__ long long div_line(long long n, long long d) {
  if (((unsigned long long)(n | d) >> 32) == 0) return (long long)((uint32_t)n / (uint32_t)d);
  return n / d;
}

// The line: every slot's tiles one behind the other, cut into one piece a warp
// of the grid: warp w of nw begins at ⌊W·w/nw⌋ (so units of equal length that
// divide the grid begin with a warp); nw ≤ W, so no piece is empty.
struct LineCut {
  long long W, nw, each, more;  // each = ⌊W/nw⌋, more = W mod nw
  __device__ __forceinline__ long long begin(long long w) const {
    return w * each + (long long)((uint32_t)more * (uint32_t)w / (uint32_t)nw);  // (both below nw < 2^16)
  }
  __device__ __forceinline__ long long of(long long at) const { return div_line((at + 1) * nw - 1, W); }  // holds `at`
};
__device__ __forceinline__ LineCut line_cut(long long W, int blocks, int warps) {
  const long long nw = max(1LL, min(W, (long long)blocks * warps)), each = div_line(W, nw);
  return LineCut{W, nw, each, W - each * nw};
}

// Where a warp's piece begins: the slot and its place on the line.
struct LinePlace {
  LineCut cut;
  long long begin, end, cum;
  int slot;
};
template <int NW>
struct LineSmem {
  long long sum[NW], cum[NW * 32];
};
// tiles(b, st) gives slot b's tiles (flagging it on st); put(b, at) is called
// once a slot, by a thread of block 0, with its place.
template <int NW, class Tiles, class Put>
__device__ __forceinline__ LinePlace line_place(int n_seqs, uint32_t* status, LineSmem<NW>& sh, Tiles&& tiles, Put&& put) {
  constexpr int NTH = NW * 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* st = blockIdx.x == 0 ? status : nullptr;
  LinePlace p{};
  long long total = 0;
  if (n_seqs > NTH) {  // several rounds: the sum first
    for (int b = tid; b < n_seqs; b += NTH) total += tiles(b, nullptr);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) sh.sum[warp] = total;
    __syncthreads();
    total = 0;
    for (int i = 0; i < NW; ++i) total += sh.sum[i];
    __syncthreads();
  }
  long long base = 0;
  for (int b0 = 0; b0 < n_seqs; b0 += NTH) {
    const int b = b0 + tid;
    const long long mine = b < n_seqs ? tiles(b, st) : 0;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) sh.sum[warp] = inc;
    __syncthreads();
    long long at = base + inc - mine, all = 0;
    for (int i = 0; i < NW; ++i) {
      if (i < warp) at += sh.sum[i];
      all += sh.sum[i];
    }
    sh.cum[tid] = at;
    if (n_seqs <= NTH) total = all;
    if (b0 == 0) {
      p.cut = line_cut(total, (int)gridDim.x, NW);
      const long long me = (long long)blockIdx.x * NW + warp;
      if (me < p.cut.nw) {
        p.begin = p.cut.begin(me);
        p.end = p.cut.begin(me + 1);
      }
    }
    if (blockIdx.x == 0 && b < n_seqs) put(b, at);
    __syncthreads();
    if (p.begin >= base && p.begin < base + all) {  // the last slot that begins at or before the piece
      int n = 0;
      for (int i = 0; i < NTH && b0 + i < n_seqs; i += 32)
        n += __popc(__ballot_sync(0xffffffffu, b0 + i + lane < n_seqs && sh.cum[i + lane] <= p.begin));
      p.slot = b0 + n - 1;
      p.cum = sh.cum[n - 1];
    }
    base += all;
    if (b0 + NTH < n_seqs) __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) put(n_seqs, total);
  return p;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

}  // namespace ekv
