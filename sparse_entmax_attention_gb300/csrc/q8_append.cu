// q8_append.cu -- the quantising append of the 8-bit paged cache, and its
// read-back.
//
// A page and KV head has one scale s for its K and one for its V rows, and a
// value is code·s. For the new rows of a page:
//   s' = max(amax/c, 2^-96, s_old),  code = nearest(x / s'),
// and when the page held rows before and s' > s_old, their codes become
// nearest(v·r), r = fl32(s_old/s'). Both roundings are of the exact quotient
// or product, ties to even: the fp32 result y is corrected to "round to odd"
// (truncated, last bit set when inexact) by the sign of its exact residual,
// and rounding that to the few bits of a code cannot round twice.
#include "q8.cuh"

namespace ekv {

constexpr float kScaleFloor = 0x1p-96f;

// y near the exact value with |error| < 1 ulp, r the sign of (exact − y):
// truncate towards zero and set the last bit when y is not exact.
__device__ __forceinline__ float to_odd(float y, float r, float sign_of) {
  uint32_t u = __float_as_uint(y);
  if (r != 0.0f) {
    if ((r < 0.0f) != (sign_of < 0.0f) && (u & 0x7fffffffu)) u -= 1u;
    u |= 1u;
  }
  return __uint_as_float(u);
}

// x/s for finite x, s ≥ 2^-96, inv ≈ 1/s: within an ulp, then to odd.
__device__ __forceinline__ float quotient_odd(float x, float s, float inv) {
  float y = x * inv;
  y = fmaf(fmaf(-y, s, x), inv, y);
  return to_odd(y, fmaf(-y, s, x), x);
}
__device__ __forceinline__ float product_odd(float v, float r) {
  const float y = v * r;
  return to_odd(y, fmaf(v, r, -y), v);
}

// Codes of two values that are already rounded to odd, in the low 16 bits.
template <bool I8>
__device__ __forceinline__ uint32_t code2(float lo, float hi) {
  if constexpr (I8) {
    const int a = min(max(__float2int_rn(lo), -127), 127), b = min(max(__float2int_rn(hi), -127), 127);
    return (uint32_t)(a & 0xff) | ((uint32_t)(b & 0xff) << 8);
  }
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

struct Q8AppendArgs {
  Q8Cache c;
  Q8Batch b;
  Q8Rows k, v;
};

// One warp per (slot, touched page, KV head, side). LPR lanes share a row,
// 8 elements (16 bytes in, 8 bytes out) each.
template <bool I8, int D>
__device__ void append_q8_page(const Q8Cache& c, const Q8Rows& rows, uint8_t* pool, float* scales, const Q8Slot& s,
                               int kvh, int lp, int lane) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, NI = 32 / RPW;  // rows a warp step, steps of the largest page
  const int P = c.P;
  const int ph = phys_page(c.block_table, s.seq, lp, c.maxp, c.nphys, lane == 0 ? c.status : nullptr);
  if (ph < 0) return;
  const int old = s.L - s.count;                       // tokens before this append
  const int n_old = max(0, old - lp * P);              // of this page
  const int hi = min(P, s.L - lp * P);
  const int r = lane / LPR, ch = lane % LPR;
  const float top = I8 ? 127.0f : 448.0f;
  const __nv_bfloat16* src = rows.p + (long long)kvh * rows.hs + ch * 8;
  uint4 x[NI];
  uint32_t am = 0u;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int t = i * RPW + r;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (t >= n_old && t < hi) x[i] = ld_stream(src + (long long)(s.start + lp * P + t - old) * rows.ts);
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) am = __vmaxu2(am, w[j] & 0x7fff7fffu);  // magnitudes order as whole numbers
  }
  uint32_t m = max(am & 0xffffu, am >> 16);
  m = __reduce_max_sync(0xffffffffu, m);
  bool odd = m >= 0x7f80u;  // an infinity or NaN among them: amax over the others
  if (odd) {
    m = 0u;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = w[j] & 0x7fffu, b = (w[j] >> 16) & 0x7fffu;
        if (a < 0x7f80u) m = max(m, a);
        if (b < 0x7f80u) m = max(m, b);
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) raise_flag(c.status, ENTMAXKV_DEV_NONFINITE);
  }
  const float amax = __uint_as_float(m << 16);
  const size_t si = (size_t)ph * c.Hkv + kvh;
  float sc = fmaxf(__fdiv_rn(amax, top), kScaleFloor);
  uint8_t* dst = pool + si * P * D + ch * 8;
  if (n_old > 0) {
    const float was = scales[si];
    if (sc > was) {
      const float ratio = __fdiv_rn(was, sc);
      for (int t = r; t < n_old; t += RPW) {
        uint2* p = reinterpret_cast<uint2*>(dst + (size_t)t * D);
        const uint2 o = *p;
        const uint32_t w[2] = {o.x, o.y};
        uint32_t y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = product_odd(code_f<I8>(w[j] >> (8 * e)), ratio);
          y[j] = code2<I8>(f[0], f[1]) | (code2<I8>(f[2], f[3]) << 16);
        }
        *p = make_uint2(y[0], y[1]);
      }
    } else {
      sc = was;
    }
  }
  const float inv = __frcp_rn(sc);
  const float lim = top * sc;  // infinities become the largest code of their sign
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int t = i * RPW + r;
    if (t < n_old || t >= hi) continue;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t y[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a = bf_lo(w[j]), b = bf_hi(w[j]);
      if (odd) {
        a = a != a ? 0.0f : fminf(fmaxf(a, -lim), lim);
        b = b != b ? 0.0f : fminf(fmaxf(b, -lim), lim);
      }
      y[j >> 1] |= code2<I8>(quotient_odd(a, sc, inv), quotient_odd(b, sc, inv)) << (16 * (j & 1));
    }
    *reinterpret_cast<uint2*>(dst + (size_t)t * D) = make_uint2(y[0], y[1]);
  }
  __syncwarp();
  if (lane == 0) scales[si] = sc;
}

// Grid: touched pages of a slot (4 warps a block), 2·KV heads, slots.
template <bool I8, int D>
__global__ void __launch_bounds__(128) append_q8_kernel(Q8AppendArgs a) {
  pdl_enter();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.y >> 1, side = blockIdx.y & 1;
  for (int b = blockIdx.z; b < a.b.n_seqs; b += gridDim.z) {
    const Q8Slot s = q8_slot(a.c, a.b, b, lane == 0 ? a.c.status : nullptr);
    if (s.count == 0) continue;
    const int first = (s.L - s.count) / a.c.P, pages = (s.L + a.c.P - 1) / a.c.P - first;
    for (int i = blockIdx.x * 4 + warp; i < pages; i += gridDim.x * 4)
      append_q8_page<I8, D>(a.c, side ? a.v : a.k, side ? a.c.v_pool : a.c.k_pool, side ? a.c.v_scale : a.c.k_scale, s,
                            kvh, first + i, lane);
  }
}

struct Q8ReadArgs {
  Q8Cache c;
  Q8Batch b;
  const int32_t* first;
  Q8Rows k, v;
};

template <bool I8, int D>
__global__ void __launch_bounds__(128) read_q8_kernel(Q8ReadArgs a) {
  pdl_enter();
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane / LPR, ch = lane % LPR;
  const int kvh = blockIdx.y >> 1, side = blockIdx.y & 1;
  const Q8Cache& c = a.c;
  const int P = c.P;
  const Q8Rows& rows = side ? a.v : a.k;
  const uint8_t* pool = side ? c.v_pool : c.k_pool;
  const float* scales = side ? c.v_scale : c.k_scale;
  for (int b = blockIdx.z; b < a.b.n_seqs; b += gridDim.z) {
    const Q8Slot s = q8_slot(c, a.b, b, lane == 0 ? c.status : nullptr);
    if (s.count == 0) continue;
    const int f = a.first[b];
    if (f < 0 || (long long)f + s.count > s.L) {
      if (lane == 0) raise_flag(c.status, ENTMAXKV_DEV_BAD_BATCH);
      continue;
    }
    const int p0 = f / P, pages = (f + s.count + P - 1) / P - p0;
    for (int i = blockIdx.x * 4 + warp; i < pages; i += gridDim.x * 4) {
      const int lp = p0 + i;
      const int ph = phys_page(c.block_table, s.seq, lp, c.maxp, c.nphys, lane == 0 ? c.status : nullptr);
      if (ph < 0) continue;
      const size_t si = (size_t)ph * c.Hkv + kvh;
      const float sc = scales[si];
      const int lo = max(0, f - lp * P), hi = min(P, f + s.count - lp * P);
      for (int t = lo + r; t < hi; t += RPW) {
        const uint2 w = *reinterpret_cast<const uint2*>(pool + (si * P + t) * D + ch * 8);
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t two = (j < 2 ? w.x : w.y) >> (16 * (j & 1));
          y[j] = bf2_rn(code_f<I8>(two) * sc, code_f<I8>(two >> 8) * sc);
        }
        *reinterpret_cast<uint4*>(rows.p + (long long)(s.start + lp * P + t - f) * rows.ts + (long long)kvh * rows.hs +
                                  ch * 8) = make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
  }
}

// Blocks over the pages that one slot can touch.
static dim3 page_grid(const Q8Cache& c, const Q8Batch& b) {
  const long long pages = min((long long)c.maxp, (long long)(b.max_count / c.P) + 2);
  return dim3((unsigned)((pages + 3) / 4), (unsigned)(2 * c.Hkv), (unsigned)b.n_seqs);
}

cudaError_t launch_append_q8(const Q8Cache& c, const Q8Batch& b, const Q8Rows& k, const Q8Rows& v, bool i8,
                             cudaStream_t st) {
  const Q8AppendArgs a{c, b, k, v};
  const dim3 grid = page_grid(c, b);
  if (i8)
    return c.D == 128 ? launch_k(false, append_q8_kernel<true, 128>, grid, dim3(128), 0, st, a)
                      : launch_k(false, append_q8_kernel<true, 64>, grid, dim3(128), 0, st, a);
  return c.D == 128 ? launch_k(false, append_q8_kernel<false, 128>, grid, dim3(128), 0, st, a)
                    : launch_k(false, append_q8_kernel<false, 64>, grid, dim3(128), 0, st, a);
}

cudaError_t launch_read_q8(const Q8Cache& c, const Q8Batch& b, const int32_t* first, const Q8Rows& k, const Q8Rows& v,
                           bool i8, cudaStream_t st) {
  const Q8ReadArgs a{c, b, first, k, v};
  const dim3 grid = page_grid(c, b);
  if (i8)
    return c.D == 128 ? launch_k(false, read_q8_kernel<true, 128>, grid, dim3(128), 0, st, a)
                      : launch_k(false, read_q8_kernel<true, 64>, grid, dim3(128), 0, st, a);
  return c.D == 128 ? launch_k(false, read_q8_kernel<false, 128>, grid, dim3(128), 0, st, a)
                    : launch_k(false, read_q8_kernel<false, 64>, grid, dim3(128), 0, st, a);
}

}  // namespace ekv
