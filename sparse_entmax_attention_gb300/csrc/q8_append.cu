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
// and rounding that to the few bits of a code cannot round twice. Eight values
// take that path only where some quotient lies near enough to a tie that the
// fp32 one could round to another code.
//
// Bound: the chain of a page from its load to its codes (about 1600 instructions a
// page, KV head and side; no pipe is full), then the bytes. A warp has one page at a time, its new rows in
// registers between the maximum and the codes, so they are read once. 32801
// tokens, 8 KV heads, d = 128, int8 (134 MB in, 67 MB out): append 47-63 us,
// read-back 38 us (5.3 TB/s); 64 sequences' single tokens: 14 us in all, of
// which the bytes are 1.2; past kPageSlots slots each warp walks the slots from the
// first (333 single tokens: append 110 us, read-back 148; 250: 8.3 and 6.2). With the exact path unrolled in the loop the append
// took 149 us, waiting for instructions.
#include "q8_tiles.cuh"

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

constexpr int kPageWarps = 8;

// The exact codes of eight bf16 values (a 16-byte word) for scale s: 8 bytes.
// `odd`: infinities become ±top·s and NaN 0 first. Out of line: it is needed
// seldom, and the loop around it is unrolled.
template <bool I8>
__device__ __noinline__ uint2 codes8_exact(uint4 x, float s, float inv, bool odd) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const float lim = (I8 ? 127.0f : 448.0f) * s;
  uint32_t y[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a = bf_lo(w[j]), b = bf_hi(w[j]);
    if (odd) {
      a = a != a ? 0.0f : fminf(fmaxf(a, -lim), lim);
      b = b != b ? 0.0f : fminf(fmaxf(b, -lim), lim);
    }
    y[j >> 1] |= code2<I8>(quotient_odd(a, s, inv), quotient_odd(b, s, inv)) << (16 * (j & 1));
  }
  return make_uint2(y[0], y[1]);
}

// The same, quickly. Whole numbers: c = the fp32 quotient x·fl(1/s) rounded is
// the right code while |x − c·s| < s/2, and that difference is exact (it is a
// multiple of s's last bit and below 2^24 of them). e4m3: the fp32 quotient is
// within 2^-22 of the exact one, relatively, so its code is the right one unless
// a border lies that near. (Borders are met often: half of a page's largest
// value is 63.5 steps, but for the rounding of s.)
template <bool I8>
__device__ __forceinline__ uint2 codes8(const uint4& x, float s, float inv, bool odd) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[2];
  bool near = odd;
  if constexpr (I8) {
    constexpr float kMagic = 12582912.0f;  // 1.5·2^23: adding it rounds to whole numbers, to even
    const unsigned long long inv2 = f2_splat(inv), mg = f2_splat(kMagic), mn = f2_splat(-kMagic), ms = f2_splat(-s);
    float far = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const unsigned long long v = f2_pack(bf_lo(w[2 * h + j]), bf_hi(w[2 * h + j]));
        const unsigned long long r = f2_fma(v, inv2, mg);
        float a, b, d0, d1;
        f2_unpack(r, a, b);
        q[2 * j] = __float_as_uint(a);
        q[2 * j + 1] = __float_as_uint(b);
        f2_unpack(f2_fma(f2_add(r, mn), ms, v), d0, d1);
        far = max3(far, fabsf(d0), fabsf(d1));
      }
      y[h] = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
    }
    near |= !(far < 0.5f * s);
  } else {
    const unsigned long long inv2 = f2_splat(inv), up = f2_splat(1.0f + 0x1p-21f), dn = f2_splat(1.0f - 0x1p-21f);
    uint32_t differ = 0u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t lo[2], hi[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const unsigned long long v = f2_mul(f2_pack(bf_lo(w[2 * h + j]), bf_hi(w[2 * h + j])), inv2);
        float a, b;
        f2_unpack(f2_mul(v, dn), a, b);
        lo[j] = code2<false>(a, b);
        f2_unpack(f2_mul(v, up), a, b);
        hi[j] = code2<false>(a, b);
      }
      y[h] = lo[0] | (lo[1] << 16);
      differ |= y[h] ^ (hi[0] | (hi[1] << 16));
    }
    near |= differ != 0u;
  }
  if (__any_sync(0xffffffffu, near)) return codes8_exact<I8>(x, s, inv, odd);
  return make_uint2(y[0], y[1]);
}

// Rows r, r + step, ... below n of a slab, D codes each, to codes of the larger
// scale: eight codes a lane.
template <bool I8>
__device__ __noinline__ void requantise(uint8_t* dst, int r, int n, int step, int D, float ratio) {
  for (int t = r; t < n; t += step) {
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
}

// One warp per (slot, touched page, KV head, side). LPR lanes share a row,
// 8 elements (16 bytes in, 8 bytes out) each; the page's new rows stay in
// registers between the maximum and the codes.
template <bool I8, int D, int P>
__device__ __forceinline__ void append_q8_page(const Q8Cache& c, const Q8Rows& rows, uint8_t* pool, float* scales,
                                               const Q8Slot& s, int kvh, int lp, int lane) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, NI = P / RPW;  // rows a warp step, steps of a page
  const int ph = phys_page(c.block_table, s.seq, lp, c.maxp, c.nphys, lane == 0 ? c.status : nullptr);
  const int old = s.L - s.count;           // tokens before this append
  const int n_old = max(0, old - lp * P);  // of this page
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
  if (ph < 0) return;
  const size_t si = (size_t)ph * c.Hkv + kvh;
  const float was = n_old > 0 ? scales[si] : 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) am = __vmaxu2(am, w[j] & 0x7fff7fffu);  // magnitudes order as whole numbers
  }
  uint32_t m = max(am & 0xffffu, am >> 16);
  m = __reduce_max_sync(0xffffffffu, m);
  const bool odd = m >= 0x7f80u;  // an infinity or NaN among them: amax over the others
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
  float sc = fmaxf(__fdiv_rn(amax, top), kScaleFloor);
  uint8_t* dst = pool + si * P * D + ch * 8;
  if (n_old > 0) {
    if (sc > was) {
      requantise<I8>(dst, r, n_old, RPW, D, __fdiv_rn(was, sc));
    } else {
      sc = was;
    }
  }
  const float inv = __frcp_rn(sc);
  if (hi - n_old == 1) {  // a decode step's token: one row
    const int i0 = n_old / RPW;
    uint4 one = x[0];
#pragma unroll
    for (int i = 1; i < NI; ++i)
      if (i == i0) one = x[i];
    const uint2 y = codes8<I8>(one, sc, inv, odd);
    if (r == n_old % RPW) *reinterpret_cast<uint2*>(dst + (size_t)n_old * D) = y;
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int t = i * RPW + r;
      const uint2 y = codes8<I8>(x[i], sc, inv, odd);
      if (t >= n_old && t < hi) *reinterpret_cast<uint2*>(dst + (size_t)t * D) = y;
    }
  }
  __syncwarp();
  if (lane == 0) scales[si] = sc;
}

// The touched pages of all slots, times KV heads and sides, form the line, and
// the grid's warps take it in turns: neighbours work on neighbouring heads of
// the same tokens. The block's first kPageSlots slots are kept at hand.
constexpr int kPageSlots = kPageWarps * 32;
template <class Find, class Work>
__device__ __forceinline__ void each_page(const Q8Cache& c, const Q8Batch& b, Find&& find, Work&& work) {
  __shared__ LineSmem<kPageWarps> sh;
  __shared__ Q8Slot slots[kPageSlots];
  __shared__ int firsts[kPageSlots];
  const int per = 2 * c.Hkv;
  const bool few = b.n_seqs <= kPageSlots;
  auto pages = [&](const Q8Slot& s, int f) { return s.count > 0 ? (f + s.count - 1) / c.P - f / c.P + 1 : 0; };
  const LinePlace at = line_place<kPageWarps>(
      b.n_seqs, c.status, sh,
      [&](int i, uint32_t* st) {
        int f;
        const Q8Slot s = find(i, f, st);
        if (few) {
          slots[i] = s;
          firsts[i] = f;
        }
        return (long long)pages(s, f) * per;
      },
      [](int, long long) {});
  const long long nw = (long long)gridDim.x * kPageWarps, W = at.cut.W;
  long long cum = 0, n = -1;
  int slot = 0, f = 0;
  Q8Slot s{-1, 0, 0, 0};
  for (long long w = (long long)blockIdx.x * kPageWarps + (threadIdx.x >> 5); w < W; w += nw) {
    if (few) {  // the last slot that begins at or before w
      int k = 0;
      for (int i = 0; i < b.n_seqs; i += 32) {
        const int j = i + (threadIdx.x & 31);
        k += __popc(__ballot_sync(0xffffffffu, j < b.n_seqs && sh.cum[j] <= w));
      }
      s = slots[k - 1];
      f = firsts[k - 1];
      cum = sh.cum[k - 1];
    } else {
      for (; n < 0 || w >= cum + n; ++slot) {
        if (n >= 0) cum += n;
        s = find(slot, f, nullptr);
        n = (long long)pages(s, f) * per;
      }
    }
    const long long u = w - cum;
    const int page = (int)div_line(u, per), rest = (int)(u - (long long)page * per);
    work(s, f, f / c.P + page, rest >> 1, rest & 1);
  }
}

template <bool I8, int D, int P>
__global__ void __launch_bounds__(kPageWarps * 32, 2) append_q8_kernel(Q8AppendArgs a) {
  pdl_enter();
  each_page(
      a.c, a.b,
      [&](int b, int& f, uint32_t* st) {
        const Q8Slot s = q8_slot(a.c, a.b, b, st);
        f = s.L - s.count;
        return s;
      },
      [&](const Q8Slot& s, int, int lp, int kvh, int side) {
        append_q8_page<I8, D, P>(a.c, side ? a.v : a.k, side ? a.c.v_pool : a.c.k_pool,
                                 side ? a.c.v_scale : a.c.k_scale, s, kvh, lp, threadIdx.x & 31);
      });
}

struct Q8ReadArgs {
  Q8Cache c;
  Q8Batch b;
  const int32_t* first;
  Q8Rows k, v;
};

template <bool I8, int D, int P>
__global__ void __launch_bounds__(kPageWarps * 32, 3) read_q8_kernel(Q8ReadArgs a) {
  pdl_enter();
  constexpr int LPR = D / 16, RPW = 32 / LPR, NI = P / RPW;  // a lane has 16 codes of a row
  const int lane = threadIdx.x & 31, r = lane / LPR, ch = lane % LPR;
  const Q8Cache& c = a.c;
  each_page(
      c, a.b,
      [&](int b, int& f, uint32_t* st) {  // count 0 where the tokens asked for are not there
        f = a.first[b];
        Q8Slot s = q8_slot(c, a.b, b, st);
        if (s.count > 0 && (f < 0 || (long long)f + s.count > s.L)) {
          raise_flag(st, ENTMAXKV_DEV_BAD_BATCH);
          s.count = 0;
        }
        return s;
      },
      [&](const Q8Slot& s, int f, int lp, int kvh, int side) {
        const Q8Rows& rows = side ? a.v : a.k;
        const int ph = phys_page(c.block_table, s.seq, lp, c.maxp, c.nphys, lane == 0 ? c.status : nullptr);
        if (ph < 0) return;
        const size_t si = (size_t)ph * c.Hkv + kvh;
        const uint8_t* src = (side ? c.v_pool : c.k_pool) + si * P * D + ch * 16;
        const int lo = max(0, f - lp * P), hi = min(P, f + s.count - lp * P);
        uint4 x[NI];
#pragma unroll
        for (int k = 0; k < NI; ++k) {
          const int t = k * RPW + r;
          x[k] = t >= lo && t < hi ? ld_stream(src + t * D) : make_uint4(0u, 0u, 0u, 0u);
        }
        const unsigned long long sc = f2_splat((side ? c.v_scale : c.k_scale)[si]);
        __nv_bfloat16* dst = rows.p + (long long)(s.start + lp * P - f) * rows.ts + (long long)kvh * rows.hs + ch * 16;
#pragma unroll
        for (int k = 0; k < NI; ++k) {
          const int t = k * RPW + r;
          const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          uint32_t y[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t h[2];
            codes_half<I8, false>(v[j], h[0], h[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
              float p, q;
              f2_unpack(f2_mul(f2_pack(g.x, g.y), sc), p, q);
              y[2 * j + e] = bf2_rn(p, q);
            }
          }
          if (t >= lo && t < hi) {
            uint4* o = reinterpret_cast<uint4*>(dst + (long long)t * rows.ts);
            o[0] = make_uint4(y[0], y[1], y[2], y[3]);
            o[1] = make_uint4(y[4], y[5], y[6], y[7]);
          }
        }
      });
}

// Blocks for the pages that a batch can touch: at most `full`, and a warp a
// page where they are few.
static int page_blocks(const Q8Cache& c, const Q8Batch& b, int full) {
  const long long items = ((long long)b.total / c.P + 2LL * b.n_seqs) * 2 * c.Hkv;
  return (int)max(1LL, min((long long)full, (items + kPageWarps - 1) / kPageWarps));
}

template <bool I8, int D>
static cudaError_t append_t(const Q8AppendArgs& a, int blocks, cudaStream_t st) {
  return a.c.P == 32 ? launch_k(true, append_q8_kernel<I8, D, 32>, dim3(blocks), dim3(kPageWarps * 32), 0, st, a)
                     : launch_k(true, append_q8_kernel<I8, D, 16>, dim3(blocks), dim3(kPageWarps * 32), 0, st, a);
}
template <bool I8, int D>
static cudaError_t read_t(const Q8ReadArgs& a, int blocks, cudaStream_t st) {
  return a.c.P == 32 ? launch_k(true, read_q8_kernel<I8, D, 32>, dim3(blocks), dim3(kPageWarps * 32), 0, st, a)
                     : launch_k(true, read_q8_kernel<I8, D, 16>, dim3(blocks), dim3(kPageWarps * 32), 0, st, a);
}

cudaError_t launch_append_q8(const Q8Cache& c, const Q8Batch& b, const Q8Rows& k, const Q8Rows& v, bool i8, int sms,
                             cudaStream_t st) {
  const Q8AppendArgs a{c, b, k, v};
  const int blocks = page_blocks(c, b, 2 * sms);
  if (i8) return c.D == 128 ? append_t<true, 128>(a, blocks, st) : append_t<true, 64>(a, blocks, st);
  return c.D == 128 ? append_t<false, 128>(a, blocks, st) : append_t<false, 64>(a, blocks, st);
}

cudaError_t launch_read_q8(const Q8Cache& c, const Q8Batch& b, const int32_t* first, const Q8Rows& k, const Q8Rows& v,
                           bool i8, int sms, cudaStream_t st) {
  const Q8ReadArgs a{c, b, first, k, v};
  const int blocks = page_blocks(c, b, 3 * sms);
  if (i8) return c.D == 128 ? read_t<true, 128>(a, blocks, st) : read_t<true, 64>(a, blocks, st);
  return c.D == 128 ? read_t<false, 128>(a, blocks, st) : read_t<false, 64>(a, blocks, st);
}

}  // namespace ekv
