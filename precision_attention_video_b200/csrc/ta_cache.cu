// ta_cache.cu -- the paged key-value cache: appending new tokens with the
// position rotation (and the mean key of every page that fills up), and the
// choice of the pages that a row reads.
#include <type_traits>

#include "ta_cache.cuh"

namespace ta {
namespace {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// One pair of a rotation: x c - y s and y c + x s.  In fp32 each operation
// rounds by itself, as an elementwise evaluation does.  In fp64 the products
// of a bf16 and an fp32 value are exact, so the result is rounded once;
// narrowed to fp32 by truncation with the last bit set when anything was cut
// off, it still rounds to any format of at most 22 bits as the exact value
// would: an FP8 code is one rounding away from the rotated key.
__device__ __forceinline__ float narrow_odd(double r) {
  const float f = __double2float_rz(r);
  return (double)f == r || !(fabsf(f) < __int_as_float(0x7f800000))
             ? f
             : __uint_as_float(__float_as_uint(f) | 1u);
}
__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
  const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = u;
}
__device__ __forceinline__ void turn_pair(float& x, float& y, double c, double s) {
  const double a = x, b = y;
  x = narrow_odd(__fma_rn(a, c, -(b * s)));
  y = narrow_odd(__fma_rn(b, c, a * s));
}

// A lane's part of the heads of one token: two chunks of 8 elements that the
// rotation pairs with each other (or within themselves), and the angles'
// cosines and sines, which serve every head of the token.  D / 16 lanes hold a
// head.
template <int D>
struct Turn {
  int eA, eB;          // first elements of the chunks
  bool on, inter;
  float c[8], s[8];
  __device__ __forceinline__ void place(int rot, bool interleaved, int pr) {
    inter = interleaved;
    on = 16 * pr < rot;
    if (on && !inter) {
      eA = 8 * pr;
      eB = eA + rot / 2;
    } else {
      eA = 16 * pr;      // (behind the rotated part, chunks pair up in order)
      eB = eA + 8;
    }
  }
  __device__ __forceinline__ void angles(const float* cos, const float* sin, int pr) {
    if (!on) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 u = *reinterpret_cast<const float4*>(cos + 8 * pr + 4 * h);
      const float4 v = *reinterpret_cast<const float4*>(sin + 8 * pr + 4 * h);
      c[4 * h] = u.x, c[4 * h + 1] = u.y, c[4 * h + 2] = u.z, c[4 * h + 3] = u.w;
      s[4 * h] = v.x, s[4 * h + 1] = v.y, s[4 * h + 2] = v.z, s[4 * h + 3] = v.w;
    }
  }
  template <typename F>    // float or double arithmetic
  __device__ __forceinline__ void apply(float (&x)[16]) const {
    if (!on) return;
    if (inter) {
#pragma unroll
      for (int i = 0; i < 8; ++i) turn_pair(x[2 * i], x[2 * i + 1], (F)c[i], (F)s[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) turn_pair(x[i], x[8 + i], (F)c[i], (F)s[i]);
    }
  }
};

__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[2 * i] = bf_lo(w[i]), x[2 * i + 1] = bf_hi(w[i]);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// Smallest power of two s >= 2^-126 with amax <= 448 s; 1 for 0, NaN when
// amax is not finite: a rotated key that passes fp32's range comes as its largest
// value (narrow_odd), which no bf16 value is.
__device__ __forceinline__ float token_scale(float amax) {
  if (amax == 0.0f) return 1.0f;
  if (!(amax < __int_as_float(0x7f7fffff))) return __int_as_float(0x7fffffff);
  int e;
  const float m = frexpf(amax, &e);   // amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
  return ldexpf(1.0f, max(m <= 0.875f ? e - 9 : e - 8, -126));
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
// Bound by memory: a token's keys and values are read once and written once.
// A block takes the new tokens of one page (of one sequence) and some key
// heads; a warp takes one token and 4 (d = 64: 8) heads at a time, a lane 16
// elements, with the token's cosines and sines in registers.  When the block's
// tokens fill the page, it reads the page's keys back (its own from L2) and
// sums them in slot order, so the mean is a function of the page alone.
constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kQueryHeads = 16;        // query heads of a warp

// Page item w -> sequence: the pages that sequence s touches get the items
// from cu[s] / page_size + 2 s on, and touch at most n / page_size + 2 pages,
// so no prefix over the sequences is needed.
__device__ __forceinline__ int item_start(const CacheArgs& a, int s) {
  return (max(a.cu[s], 0) >> a.ps_log2) + 2 * s;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kAppendThreads, 4) cache_append_kernel(const CacheArgs a, int items,
                                                                      int chunks, int hc_log2) {
  constexpr int LPH = D / 16, HPI = 32 / LPH;      // lanes of a head, heads of a warp
  constexpr int HPI_LOG2 = D == 128 ? 2 : 3;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hl = lane / LPH, pr = lane % LPH;
  const int r2 = a.rot_dim / 2;

  if ((int)blockIdx.x >= items * chunks) {
    // ---- queries: a warp takes one row and 16 heads ----
    const int hg = (a.H + kQueryHeads - 1) / kQueryHeads;
    const int w = ((int)blockIdx.x - items * chunks) * kAppendWarps + warp;
    const int t = w / hg, h0 = (w - t * hg) * kQueryHeads;
    if (t >= rows_used(a)) return;
    int p = row_pos(a, t, row_seq(a, t));
    if (p < 0) return;
    if (a.pos) p = a.pos[t];
    if (a.rot_dim && (p < 0 || p >= a.rot_rows)) {
      report_bad_index(a.status);
      return;
    }
    Turn<D> turn;
    turn.place(a.rot_dim, a.rot_interleaved, pr);
    turn.angles(a.cos + (int64_t)p * r2, a.sin + (int64_t)p * r2, pr);
    const __nv_bfloat16* q = a.q + (int64_t)t * a.sq_t;
    __nv_bfloat16* o = a.o + (int64_t)t * a.so_t;
    // each head is read and written by its own lanes: in place is fine
    constexpr int IT = kQueryHeads / HPI;
    uint4 x[IT][2];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int h = h0 + i * HPI + hl;
      if (h < a.H) {
        x[i][0] = __ldcs(reinterpret_cast<const uint4*>(q + (int64_t)h * a.sq_h + turn.eA));
        x[i][1] = __ldcs(reinterpret_cast<const uint4*>(q + (int64_t)h * a.sq_h + turn.eB));
      }
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int h = h0 + i * HPI + hl;
      if (h < a.H) {
        float y[16];
        unpack16(x[i][0], x[i][1], y);
        turn.template apply<float>(y);
        __stcs(reinterpret_cast<uint4*>(o + (int64_t)h * a.so_h + turn.eA), pack8(y));
        __stcs(reinterpret_cast<uint4*>(o + (int64_t)h * a.so_h + turn.eB), pack8(y + 8));
      }
    }
    return;
  }

  // ---- keys and values of one page ----
  const int item = blockIdx.x / chunks, h0 = (blockIdx.x - item * chunks) << hc_log2;
  int s = item, t1 = item + 1, n = 1, pj = 0;
  if (a.cu) {
    int lo = 0, hi = a.S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (item_start(a, mid) <= item) lo = mid; else hi = mid - 1;
    }
    s = lo;
    t1 = a.cu[s + 1];
    n = t1 - max(a.cu[s], 0);
    pj = item - item_start(a, s);
  }
  if (n <= 0) return;
  const int len = seq_len(a, s);
  int first = len - n;
  if (first < 0) {
    if (a.cu && threadIdx.x == 0) report_bad_index(a.status);
    first = 0;
  }
  pj += first >> a.ps_log2;
  const int p0 = max(first, pj << a.ps_log2), p1 = min(len, (pj + 1) << a.ps_log2);
  if (p0 >= p1) return;
  const int page = page_of(a, s, pj);
  if (page < 0) return;
  const int used = rows_used(a);
  const int upt = hc_log2 - HPI_LOG2;              // log2 of a token's head groups
  const int units = (p1 - p0) << upt;
  Turn<D> turn;
  turn.place(a.rot_dim, a.rot_interleaved, pr);

  for (int u = warp; u < units; u += kAppendWarps) {
    const int p = p0 + (u >> upt), h = h0 + ((u & ((1 << upt) - 1)) << HPI_LOG2) + hl;
    const int t = t1 - (len - p);
    if (t < 0 || t >= used) continue;
    const int ang = a.pos ? a.pos[t] : p;
    if (a.rot_dim && (ang < 0 || ang >= a.rot_rows)) {
      report_bad_index(a.status);
      continue;
    }
    const bool on = h < a.Hkv;
    const __nv_bfloat16* kr = a.k_new + (int64_t)t * a.sk_t + (int64_t)h * a.sk_h;
    const __nv_bfloat16* vr = a.v_new + (int64_t)t * a.sv_t + (int64_t)h * a.sv_h;
    uint4 xk[2], xv[2];
    if (on) {
      xk[0] = __ldcs(reinterpret_cast<const uint4*>(kr + turn.eA));
      xk[1] = __ldcs(reinterpret_cast<const uint4*>(kr + turn.eB));
      xv[0] = __ldcs(reinterpret_cast<const uint4*>(vr + turn.eA));
      xv[1] = __ldcs(reinterpret_cast<const uint4*>(vr + turn.eB));
    }
    turn.angles(a.cos + (int64_t)ang * r2, a.sin + (int64_t)ang * r2, pr);
    const int slot = p & (a.page_size - 1);
    const int64_t at = (int64_t)page * a.s_page + (int64_t)h * a.s_head + (int64_t)slot * a.s_slot;
    float k[16];
    if (on) {
      unpack16(xk[0], xk[1], k);
      turn.template apply<typename std::conditional<FP8, double, float>::type>(k);
    }
    if constexpr (!FP8) {
      if (on) {
        __nv_bfloat16* kd = static_cast<__nv_bfloat16*>(a.k) + at;
        __nv_bfloat16* vd = static_cast<__nv_bfloat16*>(a.v) + at;
        *reinterpret_cast<uint4*>(kd + turn.eA) = pack8(k);
        *reinterpret_cast<uint4*>(kd + turn.eB) = pack8(k + 8);
        *reinterpret_cast<uint4*>(vd + turn.eA) = xv[0];
        *reinterpret_cast<uint4*>(vd + turn.eB) = xv[1];
      }
    } else {
      // |x| as integers order like the floats, and any NaN lies above inf;
      // V's maximum comes from the packed bf16 words
      uint32_t mk = 0, mv = 0;
      if (on) {
#pragma unroll
        for (int j = 0; j < 16; ++j) mk = max(mk, __float_as_uint(k[j]) & 0x7fffffffu);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          mv = __vmaxu2(mv, __vmaxu2(__vmaxu2(xv[j].x & 0x7fff7fffu, xv[j].y & 0x7fff7fffu),
                                     __vmaxu2(xv[j].z & 0x7fff7fffu, xv[j].w & 0x7fff7fffu)));
        mv = max(mv << 16, mv & 0xffff0000u);
      }
#pragma unroll
      for (int o = 1; o < LPH; o <<= 1) {
        mk = max(mk, __shfl_xor_sync(0xffffffffu, mk, o));
        mv = max(mv, __shfl_xor_sync(0xffffffffu, mv, o));
      }
      if (on) {
        const float sk = token_scale(__uint_as_float(mk)), sv = token_scale(__uint_as_float(mv));
        const float ik = 1.0f / sk, iv = 1.0f / sv;   // powers of two: exact
        uint32_t ck[4] = {0, 0, 0, 0}, cv[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) ck[j >> 1] |= cvt_e4m3x2(k[2 * j] * ik, k[2 * j + 1] * ik) << (16 * (j & 1));
        const uint32_t w[8] = {xv[0].x, xv[0].y, xv[0].z, xv[0].w, xv[1].x, xv[1].y, xv[1].z, xv[1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) cv[j >> 1] |= cvt_e4m3x2(bf_lo(w[j]) * iv, bf_hi(w[j]) * iv) << (16 * (j & 1));
        uint8_t* kd = static_cast<uint8_t*>(a.k) + at;
        uint8_t* vd = static_cast<uint8_t*>(a.v) + at;
        *reinterpret_cast<uint2*>(kd + turn.eA) = make_uint2(ck[0], ck[1]);
        *reinterpret_cast<uint2*>(kd + turn.eB) = make_uint2(ck[2], ck[3]);
        *reinterpret_cast<uint2*>(vd + turn.eA) = make_uint2(cv[0], cv[1]);
        *reinterpret_cast<uint2*>(vd + turn.eB) = make_uint2(cv[2], cv[3]);
        if (pr == 0) {
          const int64_t so = (((int64_t)page * a.Hkv + h) << a.ps_log2) + slot;
          a.k_scale[so] = sk;
          a.v_scale[so] = sv;
        }
      }
    }
  }

  if (!a.k_mean || p1 != (pj + 1) << a.ps_log2) return;
  // ---- the page is full: its mean key, 32 lanes a head ----
  __syncthreads();
  constexpr int E = D / 32;                        // elements of a lane
  const float inv = 1.0f / (float)a.page_size;
  for (int h = h0 + warp; h < min(h0 + (1 << hc_log2), a.Hkv); h += kAppendWarps) {
    const int64_t at = (int64_t)page * a.s_page + (int64_t)h * a.s_head + E * lane;
    const float* sc = FP8 ? a.k_scale + (((int64_t)page * a.Hkv + h) << a.ps_log2) : nullptr;
    float sum[E];
#pragma unroll
    for (int j = 0; j < E; ++j) sum[j] = 0.0f;
#pragma unroll 16
    for (int r = 0; r < a.page_size; ++r) {
      float x[E];
      if constexpr (!FP8) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.k) + at + r * a.s_slot);
        uint32_t w[E / 2];
        if constexpr (E == 4) {
          const uint2 y = __ldcg(reinterpret_cast<const uint2*>(src));
          w[0] = y.x, w[1] = y.y;
        } else {
          w[0] = __ldcg(src);
        }
#pragma unroll
        for (int j = 0; j < E / 2; ++j) x[2 * j] = bf_lo(w[j]), x[2 * j + 1] = bf_hi(w[j]);
      } else {
        const uint8_t* src = static_cast<const uint8_t*>(a.k) + at + r * a.s_slot;
        uint32_t w;
        if constexpr (E == 4)
          w = __ldcg(reinterpret_cast<const uint32_t*>(src));
        else
          w = __ldcg(reinterpret_cast<const uint16_t*>(src));
        const float f = __ldcg(sc + r);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          const float2 y = e4m3x2_to_float2(w >> (16 * j));
          x[2 * j] = y.x * f;
          x[2 * j + 1] = y.y * f;
        }
      }
#pragma unroll
      for (int j = 0; j < E; ++j) sum[j] += x[j];
    }
    float* out = a.k_mean + ((int64_t)page * a.Hkv + h) * D + E * lane;
    if constexpr (E == 4)
      *reinterpret_cast<float4*>(out) = make_float4(sum[0] * inv, sum[1] * inv, sum[2] * inv, sum[3] * inv);
    else
      *reinterpret_cast<float2*>(out) = make_float2(sum[0] * inv, sum[1] * inv);
  }
}

// ---------------------------------------------------------------------------
// Choice of pages
// ---------------------------------------------------------------------------
// Per row, key head and query head g of it: logits l_gj = scale * q_g . kbar_j
// over the pages j that compete, masses M_gj = exp(l_gj - max) / sum, and the
// n_select - n_first - n_recent pages of greatest sum_g M_gj, as fp64 decides.
//
// Single rows are bound by reading the means: their logits are fp64 sums, and
// a block chooses for each (row, key head).
//
// Where many rows of a sequence share its means, fp64 would bound, and it
// decides only where it has to.  There the logits come from f16 tensor-core
// products with an fp32 sum and a bound of their error; where the last page
// that is in and the first that is out lie further apart than the bound, the
// set is the one that fp64 would find, whatever the rounding.  The other rows
// (1.6 percent on random means, and ties) are listed and done again
// in fp64.
//
// The error, in parts of |q| |kbar|, both scaled by powers of two to a largest
// element in [1, 2).  Two f16 parts hold an element of the mean to 2^-22 of it or
// half f16's smallest step, 2^-25; the query's 8 bits are exact down to 2^-17 and
// below that to 2^-25; over d = 128 elements that is 2^-22 + 2 sqrt(d) 2^-25 at
// most.  64 products each go into a sum of their own, 16 at a time with what the
// sum was, and an addend may lose 2^-24 of the largest: 4 * 17 * 2^-24 (the rest
// parts, which go first, are 2^-11 of that).  Joining the two sums and the two
// scales round by 2^-24 each.  5.15e-6 in all; what is of second order, and the
// norms' own roundings, the factor 1.1 at the decision covers.
constexpr int kSelThreads = 256;
constexpr int kSelCols = 128;          // (row, head) columns of a fast logits block
constexpr float kLogitErr = 5.2e-6f;
constexpr float kInf = 3.0e38f;        // a logit above is taken as not finite

// Pages that row t sees, and the pages [c0, c1) that compete for it.
struct RowPages {
  int n, c0, c1;
};
__device__ __forceinline__ RowPages row_pages(const CacheArgs& a, int t, int s) {
  RowPages r;
  const int len = row_pos(a, t, s) + 1;
  r.n = (len + a.page_size - 1) >> a.ps_log2;
  r.c0 = min(a.n_first, r.n);
  r.c1 = max(r.c0, r.n - a.n_recent);
  return r;
}

// Scratch.  For each (row, query head), of the rows that choose at a time,
// `pitch` doubles, of which the fp32 logits (in log2 units) take the first half
// until the row is done in fp64.
// For the fast logits also: for each (sequence, key head) the split tiles, the
// pages' norms and the powers of two that undo their scaling; the queries'
// norms; for each row its sequence and number of pages; the list of items that
// fp64 has to decide.
__device__ __forceinline__ double* logit_row(const CacheArgs& a, int t, int h) {
  return a.scratch + ((int64_t)(t - a.row0) * a.H + h) * select_pitch(a.max_pages);
}
__device__ __forceinline__ unsigned char* split_tile(const CacheArgs& a, int s, int hk, int jb, int bytes) {
  return reinterpret_cast<unsigned char*>(a.scratch + (int64_t)a.logit_rows * a.H * select_pitch(a.max_pages)) +
         (((int64_t)s * a.Hkv + hk) * (select_pitch(a.max_pages) / 128) + jb) * bytes;
}
__device__ __forceinline__ float* norm_row(const CacheArgs& a, int s, int hk) {
  return reinterpret_cast<float*>(split_tile(a, a.S, 0, 0, 512 * a.d)) + ((int64_t)s * a.Hkv + hk) * select_pitch(a.max_pages);
}
__device__ __forceinline__ float* down_row(const CacheArgs& a, int s, int hk) {
  return norm_row(a, a.S + s, hk);
}
__device__ __forceinline__ float* qnorm_row(const CacheArgs& a) { return norm_row(a, 2 * a.S, 0); }
__device__ __forceinline__ int2* row_info(const CacheArgs& a) {
  return reinterpret_cast<int2*>(qnorm_row(a) + (int64_t)(a.T + (a.T & 1)) * a.H);
}

// Items (row, key head) that fp64 has to decide, and how many.
__device__ __forceinline__ int2* again_list(const CacheArgs& a) { return row_info(a) + a.T + (a.T & 1) + 2; }
__device__ __forceinline__ int* again_count(const CacheArgs& a) { return reinterpret_cast<int*>(again_list(a) - 1); }

// A tile's rows among those that choose now.
__device__ __forceinline__ RowTile choosing_tile(const CacheArgs& a, int tile_rows) {
  RowTile r = row_tile(a, (a.cu ? a.row0 / tile_rows : a.row0) + blockIdx.x, tile_rows);
  r.t0 = max(r.t0, a.row0);
  r.t1 = min(r.t1, a.row0 + a.row_n);
  return r;
}

__device__ __forceinline__ void dmma(double (&c)[2], double a, double b) {
  asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0, %1}, {%2}, {%3}, {%0, %1};"
               : "+d"(c[0]), "+d"(c[1])
               : "d"(a), "d"(b));
}
// Two floats as f16 parts: x = hi + lo + (at most 2^-22 |x|, or 2^-25).
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
// Power of two that brings a largest magnitude x to [1, 2); 1 where x is zero,
// or not finite, or tiny: such a column's logits are made NaN, which sends
// the row to fp64.
// (unit_size is its reciprocal.)
__device__ __forceinline__ float unit_size(float x) {
  return x >= 1e-35f && x < kInf ? __uint_as_float(__float_as_uint(x) & 0x7F800000u) : 1.0f;
}
__device__ __forceinline__ float unit_scale(float x) {
  const uint32_t w = 0x7F000000u - __float_as_uint(unit_size(x));
  return __uint_as_float(w ? w : 0x00400000u);     // (2^-127 is subnormal)
}

__device__ __forceinline__ double kInf64() { return __longlong_as_double(0x7ff0000000000000ll); }
__device__ __forceinline__ bool tiny(float x) { return x > 0.0f && x < 1e-35f; }

// Place of element d in a column of fp64 queries: the two elements that a lane
// reads at a time, of its four consecutive ones, next to its neighbours'.
__device__ __forceinline__ int q_slot(int d) {
  return (d & ~15) + ((d >> 1) & 1) * 8 + ((d >> 2) & 3) * 2 + (d & 1);
}

// fp64 logits of a tile of few rows.  A warp takes 8 pages at a time, the next
// 8 on their way to shared memory: 8 lanes hold a page and multiply it with 4 columns, two
// pages for each column element read from shared memory, and 7 exchanges with
// halving leave one of the 8 sums (2 pages by 4 columns) with each lane.
template <int D>
__global__ void __launch_bounds__(kSelThreads, 3) cache_logits64_kernel(const CacheArgs a, int tile_rows,
                                                                        int pages) {
  extern __shared__ __align__(16) unsigned char sel_smem[];
  double2* qs = reinterpret_cast<double2*>(sel_smem);
  constexpr int K = D / 32, STEP = kSelThreads / 32 * 8;   // 16-byte chunks of a lane; pages of a step
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane >> 3, li = lane & 7;
  const int hk = blockIdx.y;
  const RowTile tile = choosing_tile(a, tile_rows);
  const int s = tile.s, t0 = tile.t0, t1 = tile.t1;
  if (t0 >= t1) return;
  const RowPages last = row_pages(a, t1 - 1, s);   // the tile's longest row
  const int j0 = max((int)blockIdx.z * pages, min(a.n_first, last.n));
  const int j_end = min(last.c1, (int)(blockIdx.z + 1) * pages);
  if (j0 >= j_end || last.n <= a.n_select) return;
  const int cols = (t1 - t0) * a.G, groups = (cols + 3) / 4;

  int ids = -1;                        // lane l < 8: page l of the batch after the next
  auto ask = [&](int j) {
    ids = -1;
    if (lane < 8 && j + lane < j_end) ids = page_of(a, s, j + lane);
  };
  // two batches of 8 pages for each warp, behind the queries
  float4* stage = reinterpret_cast<float4*>(qs + groups * 4 * (D / 2)) + warp * (16 * (D / 4));
  uint32_t live = 0, nlive = 0;        // pages of a batch with a mean
  auto fetch = [&](int buf, uint32_t& on) {
    on = __ballot_sync(0xffffffffu, ids >= 0);
    constexpr int PPI = 128 / D;       // pages that the warp copies at a time
#pragma unroll
    for (int i = 0; i < 8; i += PPI) {
      const int p = i + lane / (D / 4), x = lane % (D / 4);
      const int page = __shfl_sync(0xffffffffu, ids, p);
      if (page >= 0)
        cp_async16(stage + (buf * 8 + p) * (D / 4) + x, a.k_mean + ((int64_t)page * a.Hkv + hk) * D + 4 * x, 16);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int j_first = j0 + warp * 8;
  ask(j_first);
  fetch(0, live);
  ask(j_first + STEP);
  // element 4 (8 k + l) + 2 h + (0, 1) of column c at ((c K + k) 2 + h) 8 + l
  for (int i = threadIdx.x; i < groups * 4 * (D / 2); i += kSelThreads) {
    const int c = i / (D / 2), d = 2 * (i - c * (D / 2));
    double2 x = make_double2(0.0, 0.0);
    if (c < cols) {
      const int r = c / a.G, h = hk * a.G + (c - r * a.G);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(a.q + (int64_t)(t0 + r) * a.sq_t + (int64_t)h * a.sq_h + d);
      x = make_double2((double)bf_lo(w), (double)bf_hi(w));
    }
    qs[((c * K + d / 32) * 2 + (d >> 1 & 1)) * 8 + (d >> 2 & 7)] = x;
  }
  __syncthreads();
  int buf = 0;
  for (int j = j_first; j < j_end; j += STEP) {
    fetch(buf ^ 1, nlive);
    ask(j + 2 * STEP);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
    const float4* v = stage + (buf * 8 + sub) * (D / 4) + li;
    for (int c0 = 0; c0 < groups * 4; c0 += 4) {
      double w[8];                     // 4 (page) + column
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = 0.0;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        double x[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 y = v[e * D + 8 * k];
          x[e][0] = y.x, x[e][1] = y.y, x[e][2] = y.z, x[e][3] = y.w;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const double2 q0 = qs[((c0 + c) * K + k) * 16 + li], q1 = qs[((c0 + c) * K + k) * 16 + 8 + li];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            w[4 * e + c] = fma(x[e][3], q1.y, fma(x[e][2], q1.x, fma(x[e][1], q0.y, fma(x[e][0], q0.x, w[4 * e + c]))));
        }
      }
#pragma unroll
      for (int n = 4; n; n >>= 1) {    // exchange with lane ^ n, halving the sums
        const bool up = lane & n;
#pragma unroll
        for (int k = 0; k < n; ++k) {
          const double send = up ? w[k] : w[k + n], keep = up ? w[k + n] : w[k];
          w[k] = keep + __shfl_xor_sync(0xffffffffu, send, n);
        }
      }
      const int c = c0 + (li & 3), jj = j + sub + (li & 4);
      if (c < cols && jj < j_end) {
        const int r = c / a.G, h = hk * a.G + (c - r * a.G);
        logit_row(a, t0 + r, h)[jj] = live >> (sub + (li & 4)) & 1 ? w[0] * a.scale : -kInf64();
      }
    }
    live = nlive;
    buf ^= 1;
    __syncwarp();                      // all lanes have read: the buffer may be refilled
  }
}

// ---- fast logits ----
// A first kernel writes the means as tiles of 128 pages in the layout that
// the matrix instruction reads from shared memory (rows of 64 f16 elements,
// 128-byte swizzle): the leading parts, then the rest.
template <int D>
struct SplitTile {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalf = 128 * 128;          // bytes of 128 rows by 64 elements
  static constexpr int kPart = kHalves * kHalf;
  static constexpr int kBytes = 2 * kPart;
};

// Last page + 1 that any row of sequence s lets compete, 0 where no row has a
// choice to make.
__device__ __forceinline__ int pages_competing(const CacheArgs& a, int s) {
  const int t = min(a.cu[s + 1], rows_used(a)) - 1;
  if (t < max(a.cu[s], 0)) return 0;
  const RowPages r = row_pages(a, t, s);
  return r.n <= a.n_select ? 0 : r.c1;
}

template <int D>
__global__ void __launch_bounds__(kSelThreads) cache_split_kernel(const CacheArgs a) {
  using T = SplitTile<D>;
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int jb = blockIdx.x / 4, hk = blockIdx.y, s = blockIdx.z;
  const int end = pages_competing(a, s);
  if ((int)blockIdx.x * 32 >= end) return;
  unsigned char* tile = split_tile(a, s, hk, jb, T::kBytes);
  float* down = down_row(a, s, hk) + jb * 128;
  float* norm = norm_row(a, s, hk) + jb * 128;
  const int row0 = (blockIdx.x & 3) * 32 + warp * 4;
  int ids = -1;                                    // lane l < 4: the warp's page l
  {
    const int j = jb * 128 + row0 + lane;
    if (lane < 4 && j < end && j >= a.n_first) ids = page_of(a, s, j);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + i, page = __shfl_sync(0xffffffffu, ids, i);
    float x[E];
    const float* src = a.k_mean + ((int64_t)max(page, 0) * a.Hkv + hk) * D + E * lane;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = page >= 0 ? __ldg(src + e) : __int_as_float(0x7fffffff);
    float am = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) am = fmaxf(am, fabsf(x[e]));
#pragma unroll
    for (int o = 16; o; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    const float up = unit_scale(am);
    float n2 = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] *= up;
      n2 += x[e] * x[e];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
    if (lane == 0) {
      down[row] = tiny(am) ? __int_as_float(0x7fffffff) : unit_size(am);
      norm[row] = sqrtf(n2) * unit_size(am);
    }
    const int d = E * lane, half = d / 64, chunk = (d % 64) / 8;
    unsigned char* at = tile + half * T::kHalf + row * 128 + ((chunk ^ (row & 7)) << 4) + (d % 8) * 2;
    uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) split2(x[e], x[e + 1], hi[e / 2], lo[e / 2]);
    if constexpr (E == 4) {
      *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(at + T::kPart) = make_uint2(lo[0], lo[1]);
    } else {
      *reinterpret_cast<uint32_t*>(at) = hi[0];
      *reinterpret_cast<uint32_t*>(at + T::kPart) = lo[0];
    }
  }
}

// fp32 logits (in log2 units) of a tile of many rows: pages are the 128 rows of
// tcgen05.mma, the tile's (row, query head) columns its N = 128, so that a
// thread of the epilogue has one page and neighbouring threads write
// neighbouring logits.  Two sums of 64 elements each stand in TMEM (the rest
// parts' products go first, into the first of them); two blocks share an SM,
// one multiplying or loading while the other writes.
template <int D>
struct LogitsSmem {
  static constexpr int oA = 0;
  static constexpr int oB = SplitTile<D>::kBytes;
  static constexpr int oCol = oB + SplitTile<D>::kPart;      // scale and logit row of each column
  static constexpr int oBar = oCol + kSelCols * 8;
  static constexpr int kBytes = oBar + 64 + 1024;            // 1024 to align
  static constexpr int kCols = (D / 64) * kSelCols;          // TMEM columns
};

template <int D>
__global__ void __launch_bounds__(288, 2) cache_logits_kernel(const CacheArgs a, int tile_rows) {
  using T = SplitTile<D>;
  using L = LogitsSmem<D>;
  extern __shared__ unsigned char sel_raw[];
  unsigned char* smem = sel_raw + ((1024 - (smem_u32(sel_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = blockIdx.y;
  if (blockIdx.x == 0 && hk == 0 && threadIdx.x == 0) *again_count(a) = 0;
  const RowTile tile = choosing_tile(a, tile_rows);
  const int s = tile.s, t0 = tile.t0, t1 = tile.t1;
  if (t0 >= t1) return;
  if (hk == 0)
    for (int t = t0 + threadIdx.x; t < t1; t += 288) row_info(a)[t] = make_int2(s, row_pages(a, t, s).n);
  const RowPages last = row_pages(a, t1 - 1, s);   // the tile's longest row
  if (last.n <= a.n_select || last.c1 <= a.n_first) return;
  const int nb = (last.c1 + 127) / 128;
  const int cols = (t1 - t0) * a.G;
  // queries: D / 8 lanes hold a column, 8 elements each; on their way while
  // the block sets up
  constexpr int LPC = D / 8, CPB = 256 / LPC, QL = kSelCols / CPB;
  const int part = threadIdx.x % LPC;
  uint4 w[QL];
  if (warp < 8) {
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const int c = i * CPB + threadIdx.x / LPC;
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (c < cols) {
        const int r = c / a.G, h = hk * a.G + (c - r * a.G);
        w[i] = *reinterpret_cast<const uint4*>(a.q + (int64_t)(t0 + r) * a.sq_t + (int64_t)h * a.sq_h + 8 * part);
      }
    }
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::oBar);
  uint64_t *full = bars, *done = bars + 1, *freed = bars + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(bars + 3);
  int* flag = reinterpret_cast<int*>(bars + 4);
  const AbortCtx abort{flag, a.status};
  float2* col = reinterpret_cast<float2*>(smem + L::oCol);   // (scale, row as bits)

  if (threadIdx.x == 0) {
    mbar_init(full, 1);
    mbar_init(done, 1);
    mbar_init(freed, 8);
    *flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(slot, L::kCols);
    tmem_relinquish();
  }
  auto load = [&](int jb) {            // one thread: the tile of 128 pages, in 16 KB pieces
    const unsigned char* src = split_tile(a, s, hk, jb, T::kBytes);
    mbar_arrive_expect_tx(full, T::kBytes);
    for (int i = 0; i < T::kBytes; i += T::kHalf)
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
              "r"(smem_u32(smem + L::oA + i)),
          "l"(src + i), "r"(T::kHalf), "r"(smem_u32(full))
          : "memory");
  };
  __syncthreads();
  if (warp == 8 && lane == 0) load(0);
  if (warp < 8) {
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const int c = i * CPB + threadIdx.x / LPC;
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      float am = 0.0f, n2 = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) am = fmax3(am, fabsf(bf_lo(u[k])), fabsf(bf_hi(u[k])));
#pragma unroll
      for (int o = 1; o < LPC; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
      const float up = unit_scale(am);
      uint32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // (the norm of the scaled elements: a tiny query's own squares underflow)
        const float lo = bf_lo(u[k]) * up, hi = bf_hi(u[k]) * up;
        n2 += lo * lo + hi * hi;
        const __half2 z = __floats2half2_rn(lo, hi);
        y[k] = *reinterpret_cast<const uint32_t*>(&z);
      }
#pragma unroll
      for (int o = 1; o < LPC; o <<= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
      *reinterpret_cast<uint4*>(smem + L::oB + (part / 8) * T::kHalf + c * 128 + (((part % 8) ^ (c & 7)) << 4)) =
          make_uint4(y[0], y[1], y[2], y[3]);
      if (part == 0) col[c] = make_float2(am, n2);
    }
    fence_proxy_async_smem();
    // what is left of a column is one thread's (in the loop above, unrolled, it
    // was a fifth of the kernel's time, most of it in fetching instructions)
    asm volatile("bar.sync 1, 256;" ::: "memory");
    const int c = threadIdx.x;
    if (c < kSelCols) {
      const float am = col[c].x, n2 = col[c].y;
      const int r = c / a.G, row = c < cols ? r * a.H + c - r * a.G : -1;
      col[c] = make_float2(tiny(am) ? __int_as_float(0x7fffffff) : (float)(a.scale * 1.4426950408889634) * unit_size(am),
                           __int_as_float(row));
      if (row >= 0) qnorm_row(a)[(int64_t)t0 * a.H + hk * a.G + row] = sqrtf(n2) * unit_size(am);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;

  if (warp == 8) {
    if (lane == 0) {
      const uint32_t sa = smem_u32(smem + L::oA), sb = smem_u32(smem + L::oB);
      constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(kSelCols >> 3) << 17) | ((128u >> 4) << 24);   // f16 x f16
      bool ok = true;
      int i = 0;
      for (; i < nb && ok; ++i) {
        ok = mbar_wait(full, i & 1, abort, 3) && (i == 0 || mbar_wait(freed, (i - 1) & 1, abort, 4));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int part = 1; part >= 0; --part)      // the rest parts first
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t ad = smem_desc_sw128(sa + part * T::kPart + (kk >> 2) * T::kHalf + (kk & 3) * 32, 16, 1024);
            const uint64_t bd = smem_desc_sw128(sb + (kk >> 2) * T::kHalf + (kk & 3) * 32, 16, 1024);
            const bool fresh = part ? kk == 0 : (kk >= 4 && (kk & 3) == 0);
            mma_f16_ss(tmem + (part ? 0 : (kk >> 2) * kSelCols), ad, bd, idesc, fresh ? 0u : 1u);
          }
        tc_commit(done);
        ok = mbar_wait(done, i & 1, abort, 5);
        if (ok && i + 1 < nb) load(i + 1);
      }
      if (!ok) {
        // nothing may still be on its way when the block ends
        mbar_wait_drain(full, i & 1);
        mbar_wait_drain(done, i & 1);
      }
    }
  } else {
    const int64_t pitch2 = select_pitch(a.max_pages) * 2;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int c_lo = (warp >> 2) * 64, c_hi = min(cols, c_lo + 64);   // this warp's columns
    float* out = reinterpret_cast<float*>(logit_row(a, t0, hk * a.G));
    for (int i = 0; i < nb; ++i) {
      const int j = i * 128 + (threadIdx.x & 127);
      const float down = down_row(a, s, hk)[j];
      if (!mbar_wait(done, i & 1, abort, 6)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c0 = c_lo; c0 < max(c_hi, c_lo + 1); c0 += 32) {
        uint32_t x[D / 64][32];
        if constexpr (D == 128)
          tmem_ld32x2(lane_addr + c0, lane_addr + kSelCols + c0, x[0], x[1]);
        else
          tmem_ld32(lane_addr + c0, x[0]);
        if (c0 + 32 >= c_hi) {         // all read: the next product may come
          tc_fence_before();
          if (lane == 0) mbar_arrive(freed);
        }
        if (j < last.c1) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 f = col[c0 + c];
            const int row = __float_as_int(f.y);
            float y = __uint_as_float(x[0][c]);
            if (D == 128) y += __uint_as_float(x[D / 64 - 1][c]);
            if (row >= 0) out[(int64_t)row * pitch2 + j] = y * (down * f.x);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, L::kCols);
}

// Reductions over the threads of an item: one warp, or the block.
template <int WPI>
struct Group {
  float* red;                          // shared memory, 8 floats (WPI > 1)
  __device__ __forceinline__ float max(float x) const {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    if constexpr (WPI > 1) {
      __syncthreads();
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WPI; ++w) x = fmaxf(x, red[w]);
    }
    return x;
  }
  __device__ __forceinline__ float sum(float x) const {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if constexpr (WPI > 1) {
      __syncthreads();
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
      __syncthreads();
      x = red[0];
#pragma unroll
      for (int w = 1; w < WPI; ++w) x += red[w];
    }
    return x;
  }
  __device__ __forceinline__ int count(int x) const {
    x = __reduce_add_sync(0xffffffffu, x);
    if constexpr (WPI > 1) {
      __syncthreads();
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = __int_as_float(x);
      __syncthreads();
      x = 0;
#pragma unroll
      for (int w = 0; w < WPI; ++w) x += __float_as_int(red[w]);
    }
    return x;
  }
};

// Shared memory of a block's fp64 choice; reductions take turns on its halves,
// so one barrier each is enough.
constexpr int kExactHeads = 4;         // query heads taken at a time, at most
struct ExactSmem {
  double root[32];                     // 2^(k / 32)
  double red[2][kExactHeads][kSelThreads / 32];
  int cnt[2][kSelThreads / 32][4];
  uint32_t keep[kMaxSelectPages / 32];
  int key[kSelThreads];                // upper words of the threads' greatest masses
  double cand[kSelThreads];            // candidates and their pages
  int cand_j[kSelThreads];
  int cut, n_cand;
};
struct Block64 {
  ExactSmem& sm;
  int turn = 0;
  template <int N, typename Op>
  __device__ __forceinline__ void reduce(double (&x)[N], Op op) {
    double (*r)[kSelThreads / 32] = sm.red[turn ^= 1];
#pragma unroll 1
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = op(x[k], __shfl_xor_sync(0xffffffffu, x[k], o));
#pragma unroll
    for (int k = 0; k < N; ++k)
      if ((threadIdx.x & 31) == 0) r[k][threadIdx.x >> 5] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      x[k] = r[k][0];
#pragma unroll
      for (int w = 1; w < kSelThreads / 32; ++w) x[k] = op(x[k], r[k][w]);
    }
  }
  __device__ __forceinline__ void count(int (&x)[3]) {
    int (*r)[4] = sm.cnt[turn ^= 1];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      x[k] = __reduce_add_sync(0xffffffffu, x[k]);
      if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5][k] = x[k];
    }
    __syncthreads();
    x[0] = x[1] = x[2] = 0;
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w)
#pragma unroll
      for (int k = 0; k < 3; ++k) x[k] += r[w][k];
  }
};

// e^x for x <= 0, to about one unit in the last place: x = (32 e + k) ln2 / 32 + r,
// 2^e 2^(k/32) (1 + r + r^2/2 + ... + r^6/720), with Cody and Waite's reduction
// and Tang's table; the series' rest is 4e-18 of it.  Without a branch, so that
// a thread's several run side by side (calls of exp took their turns).
__device__ __forceinline__ double exp_down(const double* root, double x) {
  const double magic = 6755399441055744.0;         // 1.5 * 2^52: the sum's low bits are the integer
  const double y = fmax(x, -900.0);                // (0 below -745)
  const double z = fma(y, 46.166241308446828384, magic), n = z - magic;
  const int k = __double2loint(z), e = k >> 5;
  double r = fma(n, -0x1.62e42feep-6, y);          // ln2 / 32 in two parts, the first of 32 bits
  r = fma(n, -0x1.a39ef35793c76p-38, r);
  double p = fma(r, 1.0 / 720.0, 1.0 / 120.0);
  p = fma(r, p, 1.0 / 24.0);
  p = fma(r, p, 1.0 / 6.0);
  p = fma(r, p, 0.5);
  p = fma(r, p, 1.0);
  const double t = root[k & 31], v = fma(t * r, p, t);
  const int e1 = e >> 1;                           // (two steps: the result may be subnormal)
  return v * __hiloint2double((1023 + e1) << 20, 0) * __hiloint2double((1023 + e - e1) << 20, 0);
}

// The choice of one item from its fp64 logits, by the whole block.  x: room for
// the logits of HN query heads, which hold those of all of them already
// (`there`) or come from the item's scratch rows; the masses take the first one's
// place.  The code runs once or twice in a block's life, so its loops stay rolled:
// unrolled over a thread's pages, fetching instructions took half the time.
template <int HN>
__device__ __forceinline__ void choose64(const CacheArgs& a, int t, int hk, const RowPages r, ExactSmem& sm,
                                      double* x, bool there) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* sel = a.sel + ((int64_t)t * a.Hkv + hk) * a.n_select;
  const int nc = r.c1 - r.c0, pitch = (int)select_pitch(a.max_pages);
  const int want = a.n_select - a.n_first - a.n_recent;
  Block64 blk{sm};
  auto larger = [](double x, double y) { return fmax(x, y); };
  auto plus = [](double x, double y) { return x + y; };

  // ---- masses: a thread has pages tid + 256 i ----
  if (tid < 32) sm.root[tid] = exp2(tid * 0.03125);        // (read behind the first reduction's barrier)
  double top = -1.0;
  double* all = logit_row(a, t, hk * a.G) + r.c0;          // masses between two sets of heads
  for (int g0 = 0; g0 < a.G; g0 += HN) {
    const int nh = min(HN, a.G - g0);
    if (!there) {
      const double* l = logit_row(a, t, hk * a.G + g0) + r.c0;
#pragma unroll 4
      for (int j = tid; j < nc; j += kSelThreads)
#pragma unroll
        for (int h = 0; h < HN; ++h)
          if (h < nh) cp_async8(x + h * pitch + j, l + (int64_t)h * pitch + j);
      cp_async_wait_all();
    }
    double mx[HN], sum[HN], inv[HN];
#pragma unroll
    for (int h = 0; h < HN; ++h) mx[h] = -kInf64(), sum[h] = 0.0;
    // (a head behind the last one: x holds anything there, which nothing uses)
#pragma unroll 2
    for (int j = tid; j < nc; j += kSelThreads)
#pragma unroll
      for (int h = 0; h < HN; ++h) {
        const double y = x[h * pitch + j];
        mx[h] = isfinite(y) && y > mx[h] ? y : mx[h];
      }
    blk.reduce(mx, larger);                        // (-inf: a head without a finite logit)
#pragma unroll(4 / HN)
    for (int j = tid; j < nc; j += kSelThreads)
#pragma unroll
      for (int h = 0; h < HN; ++h) {
        const double y = x[h * pitch + j], e = exp_down(sm.root, y - mx[h]), z = isfinite(y) ? e : 0.0;
        x[h * pitch + j] = z;
        sum[h] += z;
      }
    blk.reduce(sum, plus);
#pragma unroll
    for (int h = 0; h < HN; ++h) inv[h] = h < nh && sum[h] > 0.0 ? 1.0 / sum[h] : 0.0;
    const bool last = g0 + HN >= a.G;
#pragma unroll 2
    for (int j = tid; j < nc; j += kSelThreads) {
      double m = g0 ? all[j] : 0.0;
#pragma unroll
      for (int h = 0; h < HN; ++h)
        if (h < nh) m = fma(x[h * pitch + j], inv[h], m);
      if (last) {
        x[j] = m;
        top = m > top ? m : top;
      } else {
        all[j] = m;
      }
    }
  }

  const int words = (nc + 31) / 32;
  for (int w = tid; w < words; w += kSelThreads) sm.keep[w] = 0;
  // ---- candidates: a value that `want` of the threads' greatest masses reach
  // (in their upper words, which order as they do: masses are not negative),
  // and hardly more, is one that everything kept reaches ----
  sm.key[tid] = __double2hiint(top);
  if (tid == 0) sm.n_cand = 0;
  __syncthreads();
  if (warp == 0) {
    int k[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = sm.key[lane + 32 * i];
    int hi = k[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) hi = max(hi, k[i]);
    hi = __reduce_max_sync(0xffffffffu, hi) + 1;
    int lo = 0;                                    // count(>= lo) >= want > count(>= hi)
    while (hi - lo > 1) {
      // three cuts a pass, their counts (256 at most) in one sum
      const int step = max((hi - lo) >> 2, 1), c1 = lo + step, c2 = c1 + step, c3 = c2 + step;
      int n = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) n += (k[i] >= c1) + ((k[i] >= c2) << 10) + ((k[i] >= c3) << 20);
      n = __reduce_add_sync(0xffffffffu, n);
      const int n1 = n & 1023, n2 = n >> 10 & 1023, n3 = n >> 20;
      if (n1 < want) {
        hi = c1;
        continue;
      }
      lo = n3 >= want ? c3 : n2 >= want ? c2 : c1;
      hi = n3 >= want ? hi : min(hi, lo + step);
      if ((n3 >= want ? n3 : n2 >= want ? n2 : n1) <= want + 16) break;
    }
    if (lane == 0) sm.cut = lo;
  }
  __syncthreads();
  const int cut = sm.cut;
#pragma unroll 1
  for (int j = tid; j < nc; j += kSelThreads) {
    const double m = x[j];
    if (__double2hiint(m) < cut) continue;
    const int at = atomicAdd(&sm.n_cand, 1);
    if (at < kSelThreads) {
      sm.cand[at] = m;
      sm.cand_j[at] = j;
    }
  }
  __syncthreads();
  const int n_cand = sm.n_cand;
  if (n_cand >= want && n_cand <= kSelThreads) {
    // a candidate's rank by (-mass, page) settles it (whatever the order in
    // which the candidates came)
    if (tid < n_cand) {
      // (as bits, which order as the masses do)
      const long long m = __double_as_longlong(sm.cand[tid]);
      const int j = sm.cand_j[tid];
      int rank = 0;
#pragma unroll 8
      for (int k = 0; k < n_cand; ++k) {
        const long long o = __double_as_longlong(sm.cand[k]);
        const int oj = sm.cand_j[k];
        rank += (int)(o > m) | ((int)(o == m) & (int)(oj < j));
      }
      if (rank < want) atomicOr(&sm.keep[j >> 5], 1u << (j & 31));
    }
  } else {
    // too many to rank (more than 256 places, or many equal masses): the
    // want-th greatest mass, by bisection on the bits
    double all_top[1] = {top};
    blk.reduce(all_top, larger);
    long long lo = 0, hi = __double_as_longlong(all_top[0]) + 1;   // count(>= lo) > want > count(>= hi)
    int above = 0;                                          // count(>= hi)
    while (hi - lo > 1) {
      // three cuts a pass: a barrier costs more than the comparisons
      const long long step = max((hi - lo) >> 2, 1ll);
      int n[3] = {0, 0, 0};
#pragma unroll 1
      for (int j = tid; j < nc; j += kSelThreads) {
        const long long b = __double_as_longlong(x[j]);
#pragma unroll
        for (int k = 0; k < 3; ++k) n[k] += b >= lo + (k + 1) * step;
      }
      blk.count(n);
      bool done = false;
      long long nlo = lo, nhi = hi;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const long long cut = lo + (k + 1) * step;
        if (cut >= hi || done) continue;
        if (n[k] == want) {
          nlo = nhi = cut;
          above = want;
          done = true;
        } else if (n[k] > want) {
          nlo = cut;
        } else if (cut < nhi) {
          nhi = cut;
          above = n[k];
        }
      }
      lo = nlo;
      hi = nhi;
    }
    // kept: every mass >= hi, and of those equal to lo (ties) the first ones
    int ties = want - above;
#pragma unroll 1
    for (int first = 0; first < nc; first += kSelThreads) {
      const long long b = first + tid < nc ? __double_as_longlong(x[first + tid]) : -1;
      bool keep = b >= hi;
      if (ties > 0) {                                       // uniform
        const bool eq = b == lo && b < hi;
        const uint32_t be = __ballot_sync(0xffffffffu, eq);
        int (*r2)[4] = sm.cnt[blk.turn ^= 1];
        if (lane == 0) r2[warp][0] = __popc(be);
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kSelThreads / 32; ++w) {
          if (w < warp) before += r2[w][0];
          all += r2[w][0];
        }
        keep |= eq && before + __popc(be & ((1u << lane) - 1)) < ties;
        ties -= min(ties, all);
      }
      const uint32_t bk = __ballot_sync(0xffffffffu, keep);
      if (lane == 0) sm.keep[first / 32 + warp] = bk;
    }
  }
  __syncthreads();
  // ---- the list, in page order ----
  if (warp == 0) {
    const int per = (words + 31) / 32;
    int n = 0;
    for (int k = 0; k < per; ++k)
      if (lane * per + k < words) n += __popc(sm.keep[lane * per + k]);
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    int at = a.n_first + inc - n;
    for (int k = 0; k < per; ++k) {
      if (lane * per + k >= words) break;
      uint32_t w = sm.keep[lane * per + k];
      while (w) {
        const int b = __ffs(w) - 1;
        w &= w - 1;
        if (at < a.n_select - a.n_recent) sel[at++] = r.c0 + (lane * per + k) * 32 + b;
      }
    }
  }
}

// The fixed pages of a row's list, or the whole list where every page fits;
// true where pages compete for places.
__device__ __forceinline__ bool fixed_pages(const CacheArgs& a, const RowPages& r, int64_t item, int id,
                                            int step) {
  int* sel = a.sel + item * a.n_select;
  if (r.n <= a.n_select) {
    for (int i = id; i < a.n_select; i += step) sel[i] = i < r.n ? i : -1;
    return false;
  }
  for (int i = id; i < a.n_first; i += step) sel[i] = i;
  for (int i = id; i < a.n_recent; i += step) sel[a.n_select - a.n_recent + i] = r.c1 + i;
  return a.n_select > a.n_first + a.n_recent;
}

template <int HN>
__global__ void __launch_bounds__(kSelThreads, 3) cache_choose64_kernel(const CacheArgs a) {
  __shared__ ExactSmem sm;
  extern __shared__ __align__(16) unsigned char sel_smem[];
  const int t = a.row0 + blockIdx.x, hk = blockIdx.y;
  if (t >= rows_used(a)) return;
  const RowPages r = row_pages(a, t, row_seq(a, t));
  if (fixed_pages(a, r, (int64_t)t * a.Hkv + hk, threadIdx.x, kSelThreads))
    choose64<HN>(a, t, hk, r, sm, reinterpret_cast<double*>(sel_smem), false);
}

// fp64 logits of one item by the whole block: into x, or without it into the
// item's scratch rows.
template <int D>
__device__ __forceinline__ void logits64_item(const CacheArgs& a, int t, int hk, int s, const RowPages r, double* qs,
                                           double* x) {
  constexpr int QP = D + 8;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tg = lane & 3;
  const int64_t pitch = select_pitch(a.max_pages);
  double* out = x ? x - r.c0 : logit_row(a, t, hk * a.G);
  for (int g0 = 0; g0 < a.G; g0 += 8) {
    __syncthreads();
    for (int i = tid; i < 8 * D; i += kSelThreads) {
      const int c = i / D, d = i - c * D;
      qs[c * QP + q_slot(d)] = g0 + c < a.G ? (double)__bfloat162float(a.q[(int64_t)t * a.sq_t + (int64_t)(hk * a.G + g0 + c) * a.sq_h + d]) : 0.0;
    }
    __syncthreads();
    for (int j = r.c0 + warp * 8; j < r.c1; j += kSelThreads / 32 * 8) {
      const int page = j + g < r.c1 ? page_of(a, s, j + g) : -1;
      const float4* src = reinterpret_cast<const float4*>(a.k_mean + ((int64_t)max(page, 0) * a.Hkv + hk) * D);
      float4 v[D / 16];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) v[i] = page >= 0 ? __ldg(src + 4 * i + tg) : make_float4(0.f, 0.f, 0.f, 0.f);
      double c0[2] = {0.0, 0.0}, c1[2] = {0.0, 0.0}, c2[2] = {0.0, 0.0}, c3[2] = {0.0, 0.0};
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const double* q = qs + g * QP + 2 * tg + 16 * i;
        const double2 x = *reinterpret_cast<const double2*>(q);
        const double2 y = *reinterpret_cast<const double2*>(q + 8);
        dmma(c0, v[i].x, x.x);
        dmma(c1, v[i].y, x.y);
        dmma(c2, v[i].z, y.x);
        dmma(c3, v[i].w, y.y);
      }
      if (j + g < r.c1) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (g0 + 2 * tg + e < a.G)
            out[(g0 + 2 * tg + e) * pitch + j + g] = page < 0 ? -kInf64() : ((c0[e] + c1[e]) + (c2[e] + c3[e])) * a.scale;
      }
    }
  }
  __syncthreads();
}

// Shared memory of the fast choice.
template <int WPI, int E>
struct FastSmem {
  float red[kSelThreads / 32];
  uint32_t bits[WPI > 1 ? WPI * E : 1];
  float few_mass[WPI == 1 ? 8 : 1][64];
};

// WPI warps choose for one (row, key head) of sequence s, each thread holding
// E of its pages; true where fp64 has to decide.
template <int WPI, int E, class Smem>
__device__ __forceinline__ bool fast_choice(const CacheArgs& a, Smem& sm, int t, int hk, int s, const RowPages& r,
                                            int* sel) {
  constexpr int GS = 32 * WPI;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lid = WPI == 1 ? lane : threadIdx.x;           // thread of the item
  const Group<WPI> grp{sm.red};
  const int nc = r.c1 - r.c0, want = a.n_select - a.n_first - a.n_recent;
  bool again = false;
  float mass[E];
#pragma unroll
  for (int i = 0; i < E; ++i) mass[i] = 0.0f;
  // thread's pages lid + GS i, i < mine
  const int mine_n = lid < nc ? (nc - lid + GS - 1) / GS : 0;
  float kn = 0.0f, qn = 0.0f;
  const float* nr = norm_row(a, s, hk) + r.c0 + lid;
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (i < mine_n) kn = fmaxf(kn, nr[GS * i]);
  kn = grp.max(kn);
  bool bad = false;
  const int64_t lstep = select_pitch(a.max_pages) * 2;
  const float* l = reinterpret_cast<const float*>(logit_row(a, t, hk * a.G)) + r.c0 + lid;
  float nx[E];                                         // the next head's logits
#pragma unroll
  for (int i = 0; i < E; ++i) nx[i] = i < mine_n ? l[GS * i] : -kInf;
  for (int gq = 0; gq < a.G; ++gq) {
    qn = fmaxf(qn, qnorm_row(a)[(int64_t)t * a.H + hk * a.G + gq]);
    float x[E], mx = -kInf;
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = nx[i];
    if (gq + 1 < a.G) {
      l += lstep;
#pragma unroll
      for (int i = 0; i < E; ++i) nx[i] = i < mine_n ? l[GS * i] : -kInf;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) mx = fmaxf(mx, x[i]);
    mx = grp.max(mx);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x[i]) : "f"(x[i] - mx));
      sum += x[i];
    }
    sum = grp.sum(sum);
    bad |= !(sum >= 0.5f && mx < kInf);                // a logit that is not finite
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < E; ++i) mass[i] = fmaf(x[i], inv, mass[i]);
  }
  bad |= !(kn * qn < kInf);                            // (all of these uniform)
  float top = -1.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (i >= mine_n) mass[i] = -1.0f;
    top = fmaxf(top, mass[i]);
  }
  // a float that `want` masses reach and the others do not: by bisection
  // on the bits; count(>= lo) >= want >= count(>= hi)
  int cut = -1;
  if (!bad) {
    int lo = 0, hi;
    bool few = false;                                  // only few masses lie above lo
    if (WPI == 1 && want <= 32) {
      // the want-th greatest of the lanes' greatest: it and everything
      // above it are `want` masses or more, and hardly more
      int up = __float_as_int(__uint_as_float(__reduce_max_sync(0xffffffffu, max(__float_as_int(top), 0)))) + 1;
      hi = up;
      while (up - lo > 1) {
        const int mid = lo + ((up - lo) >> 1);
        const int n = __popc(__ballot_sync(0xffffffffu, __float_as_int(top) >= mid));
        if (n >= want) lo = mid; else up = mid;
        if (n == want) break;
      }
      // its survivors, up to two a lane
      int n = 0;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const uint32_t b = __ballot_sync(0xffffffffu, __float_as_int(mass[i]) >= lo);
        const int at = n + __popc(b & ((1u << lane) - 1));
        if (__float_as_int(mass[i]) >= lo && at < 64) sm.few_mass[warp][at] = mass[i];
        n += __popc(b);
      }
      few = n <= 64;
      if (few) {
        __syncwarp();
        const int m0 = lane < n ? __float_as_int(sm.few_mass[warp][lane]) : -1;
        const int m1 = lane + 32 < n ? __float_as_int(sm.few_mass[warp][lane + 32]) : -1;
        if (n == want) cut = lo;
        while (cut < 0 && hi - lo > 1) {
          const int mid = lo + ((hi - lo) >> 1);
          const int k = __popc(__ballot_sync(0xffffffffu, m0 >= mid)) + __popc(__ballot_sync(0xffffffffu, m1 >= mid));
          if (k == want) cut = mid;
          if (k > want) lo = mid; else hi = mid;
        }
      }
    } else {
      hi = __float_as_int(grp.max(top)) + 1;
    }
    while (!few && hi - lo > 1) {
      const int mid = lo + ((hi - lo) >> 1);
      int n = 0;
#pragma unroll
      for (int i = 0; i < E; ++i) n += __float_as_int(mass[i]) >= mid;
      n = grp.count(n);
      if (n == want) {
        cut = mid;
        break;
      }
      if (n > want) lo = mid; else hi = mid;
    }
  }
  if (cut < 0) {
    again = true;                                      // equal floats, or values not finite
  } else {
    const float c = __int_as_float(cut);
    float in = kInf, out = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (mass[i] >= c) in = fminf(in, mass[i]); else out = fmaxf(out, mass[i]);
    }
    in = -grp.max(-in);
    out = grp.max(out);
    // relative error of a mass: the logits' error in the exponent of the
    // term and of the sum, ex2 and its argument (near the border up to
    // ln(1 / mass) below the maximum), and the sums' roundings
    const float delta = kLogitErr * (float)a.scale * qn * kn;
    const float err = 2.0f * delta + 1.2e-7f * (float)(E + 26 + a.G) + 4.8e-7f * (8.0f - logf(fmaxf(out, 1e-37f)));
    // and what a mass may lack outright: a head's term below 2^-126 counts as
    // 0 (a head's sum is 1 at least, so its share of the mass is no larger), and
    // sums down there round by 2^-150
    const float lost = 2.36e-38f * (float)a.G;             // 2^-125 a head
    again = !(delta < 0.05f) || !(in * (1.0f - 1.1f * err) > out * (1.0f + 1.1f * err) + lost);
    if (!again) {
      uint32_t mine = 0;                               // WPI = 1: word `lane`
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const uint32_t b = __ballot_sync(0xffffffffu, mass[i] >= c);
        if constexpr (WPI == 1) {
          if (lane == i) mine = b;
        } else {
          if (lane == 0) sm.bits[i * WPI + warp] = b;
        }
      }
      constexpr int WPL = WPI == 1 ? 1 : (WPI * E + 31) / 32;   // words of a lane
      if constexpr (WPI > 1) __syncthreads();
      if (WPI == 1 || warp == 0) {
        uint32_t w[WPL];
        int n = 0;
#pragma unroll
        for (int k = 0; k < WPL; ++k) {
          w[k] = WPI == 1 ? mine : (lane * WPL + k < WPI * E ? sm.bits[lane * WPL + k] : 0u);
          n += __popc(w[k]);
        }
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        int at = a.n_first + inc - n;
#pragma unroll
        for (int k = 0; k < WPL; ++k)
          while (w[k]) {
            const int b = __ffs(w[k]) - 1;
            w[k] &= w[k] - 1;
            sel[at++] = r.c0 + (lane * WPL + k) * 32 + b;
          }
      }
    }
  }
  return again;
}

// A block has 8 / WPI items.  Rows with half the pages or fewer take half the
// registers' steps.
template <int WPI, int E>
__global__ void __launch_bounds__(kSelThreads, E == 16 ? 4 : E == 32 ? 2 : 1) cache_choose_kernel(const CacheArgs a) {
  __shared__ FastSmem<WPI, E> sm;
  constexpr int IPB = 8 / WPI, GS = 32 * WPI;
  const int warp = threadIdx.x >> 5, lid = WPI == 1 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t item = (int64_t)a.row0 * a.Hkv + (int64_t)blockIdx.x * IPB + (WPI == 1 ? warp : 0);
  const int t = (int)(item / a.Hkv), hk = (int)(item - (int64_t)t * a.Hkv);
  if (t >= min(rows_used(a), a.row0 + a.row_n)) return;
  const int2 info = row_info(a)[t];
  // (a row that a malformed cu gives to no tile has none: no pages)
  const bool known = (unsigned)info.x < (unsigned)a.S && (unsigned)info.y <= (unsigned)a.max_pages;
  RowPages r;
  r.n = known ? info.y : 0;
  r.c0 = min(a.n_first, r.n);
  r.c1 = max(r.c0, r.n - a.n_recent);
  if (!fixed_pages(a, r, item, lid, GS)) return;           // 0 < want < nc
  int* sel = a.sel + item * a.n_select;
  const bool again = r.c1 - r.c0 <= GS * E / 2 ? fast_choice<WPI, E / 2>(a, sm, t, hk, info.x, r, sel)
                                               : fast_choice<WPI, E>(a, sm, t, hk, info.x, r, sel);
  if (again && lid == 0) again_list(a)[atomicAdd(again_count(a), 1)] = make_int2(t, hk);
}

// The items that the fast choice left, a block each at a time.
template <int D, int HN>
__global__ void __launch_bounds__(kSelThreads, 3) cache_again_kernel(const CacheArgs a) {
  __shared__ __align__(16) double qs[8 * (D + 8)];
  __shared__ ExactSmem sm;
  extern __shared__ __align__(16) unsigned char sel_smem[];
  double* x = reinterpret_cast<double*>(sel_smem);
  const int n = *again_count(a);
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int2 it = again_list(a)[i], info = row_info(a)[it.x];
    RowPages r;
    r.n = info.y;
    r.c0 = min(a.n_first, r.n);
    r.c1 = max(r.c0, r.n - a.n_recent);
    const bool fits = a.G <= HN;
    logits64_item<D>(a, it.x, it.y, info.x, r, qs, fits ? x : nullptr);
    choose64<HN>(a, it.x, it.y, r, sm, x, fits);
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_cache_append(const CacheArgs& a, cudaStream_t s) {
  const int64_t items = a.cu ? (int64_t)(a.T >> a.ps_log2) + 2 * (int64_t)a.S : a.S;
  // heads of a block: eight warps' worth where each block has one token;
  // with more tokens fewer, down to one warp's, until every SM has blocks
  const int hpi_log2 = a.d == 128 ? 2 : 3;
  int hc_log2 = hpi_log2 + 3;
  auto chunks_of = [&](int hc) { return (int64_t)((a.Hkv + (1 << hc) - 1) >> hc); };
  while (hc_log2 > hpi_log2 &&
         (chunks_of(hc_log2 - 1) == 1 || (a.cu && items * chunks_of(hc_log2) < 592)))
    --hc_log2;
  const int64_t chunks = chunks_of(hc_log2);
  const int64_t hg = (a.H + kQueryHeads - 1) / kQueryHeads;
  const int64_t qblocks = a.q ? ((int64_t)a.T * hg + kAppendWarps - 1) / kAppendWarps : 0;
  const int64_t grid = items * chunks + qblocks;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    kernel<<<(int)grid, kAppendThreads, 0, s>>>(a, (int)items, (int)chunks, hc_log2);
    return cudaGetLastError();
  };
  if (a.d == 128) return a.fp8 ? go(cache_append_kernel<128, true>) : go(cache_append_kernel<128, false>);
  return a.fp8 ? go(cache_append_kernel<64, true>) : go(cache_append_kernel<64, false>);
}

// A kernel of the fp64 choice (ID: one for each, for its shared-memory limit).
template <int ID, typename Kernel>
static cudaError_t run_exact(Kernel k, dim3 grid, int bytes, int dev, const CacheArgs& a, cudaStream_t s) {
  static OncePerDevice once;
  const cudaError_t e = once.allow(reinterpret_cast<const void*>(k), dev, kMaxSelectPages * 8);
  if (e != cudaSuccess) return e;
  k<<<grid, kSelThreads, bytes, s>>>(a);
  return cudaGetLastError();
}

template <int D>
static cudaError_t select_d(CacheArgs a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(dev, sms);
  if (e != cudaSuccess) return e;
  a.logit_rows = select_rows(a.H, a.T, a.max_pages);
  // The fast logits (a key head's queries have to fit a tile) take four kernels,
  // 28 us for a row and for a hundred; fp64 takes two, whose time grows with the
  // rows: 8 key heads of 4 query heads over 160 pages, 63 rows: 35 us fast and
  // 24 in fp64, 158 rows: 36 and 45; 4 key heads of 1 over 140 pages, 158 rows:
  // 29 and 20, 904 rows: 38 and 63.
  const bool fast = a.cu && rows_share_means(a.T, a.S) && a.G <= kSelCols &&
                    (int64_t)a.T * a.Hkv * (a.G > 1 ? a.G : 2) >= 20ll * sms;
  const int most = fast ? kSelCols : 8;
  const int tile_rows = !a.cu || a.G >= most ? 1 : most / a.G;
  static OncePerDevice once_f, once_d;
  if (fast) {
    cache_split_kernel<D><<<dim3((unsigned)(select_pitch(a.max_pages) / 32), a.Hkv, a.S), kSelThreads, 0, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = once_f.allow(reinterpret_cast<const void*>(cache_logits_kernel<D>), dev, LogitsSmem<D>::kBytes);
  } else {
    e = once_d.allow(reinterpret_cast<const void*>(cache_logits64_kernel<D>), dev, 232448);
  }
  if (e != cudaSuccess) return e;
  // the fp64 choice: so many heads' logits in shared memory that three blocks
  // share an SM
  int heads = kExactHeads;
  while (heads > 1 && (heads / 2 >= a.G || heads * select_pitch(a.max_pages) * 8 > 65536)) heads /= 2;
  const int exact = heads * (int)select_pitch(a.max_pages) * 8;
  for (a.row0 = 0; a.row0 < a.T; a.row0 += a.logit_rows) {
    a.row_n = a.logit_rows < a.T - a.row0 ? a.logit_rows : a.T - a.row0;
    // tiles that hold these rows: row t of sequence s > 0 lies in tile
    // t / tile_rows + s or in the one before, of sequence 0 in t / tile_rows
    const int64_t tiles = a.cu ? (int64_t)((a.row0 + a.row_n - 1) / tile_rows - a.row0 / tile_rows) + a.S : a.row_n;
    const int64_t items = (int64_t)a.row_n * a.Hkv;
    if (fast) {
      cache_logits_kernel<D><<<dim3((unsigned)tiles, a.Hkv), 288, LogitsSmem<D>::kBytes, s>>>(a, tile_rows);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      if (a.max_pages <= 512) {
        cache_choose_kernel<1, 16><<<(unsigned)((items + 7) / 8), kSelThreads, 0, s>>>(a);
      } else if (a.max_pages <= 1024) {
        cache_choose_kernel<1, 32><<<(unsigned)((items + 7) / 8), kSelThreads, 0, s>>>(a);
      } else if (a.max_pages <= 8192) {
        cache_choose_kernel<8, 32><<<(unsigned)items, kSelThreads, 0, s>>>(a);
      } else {
        cache_choose_kernel<8, 64><<<(unsigned)items, kSelThreads, 0, s>>>(a);
      }
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      const dim3 again((unsigned)(items < 4ll * sms ? items : 4ll * sms));
      e = heads == 4   ? run_exact<10 * D + 4>(cache_again_kernel<D, 4>, again, exact, dev, a, s)
          : heads == 2 ? run_exact<10 * D + 2>(cache_again_kernel<D, 2>, again, exact, dev, a, s)
                       : run_exact<10 * D + 1>(cache_again_kernel<D, 1>, again, exact, dev, a, s);
    } else {
      // pages of a block: all of them, or so few that every SM has blocks, a
      // multiple of what a block's warps take at a time
      const int step = 64, groups = (tile_rows * a.G + 3) / 4;
      int pages = (a.max_pages + step - 1) / step * step;
      while (pages > 2 * step && tiles * a.Hkv * ((a.max_pages + pages - 1) / pages) < 8ll * sms)
        pages = (pages / 2 + step - 1) / step * step;
      const int bytes = groups * 4 * D * 8 + kSelThreads / 32 * 16 * D * 4;
      cache_logits64_kernel<D><<<dim3((unsigned)tiles, a.Hkv, (a.max_pages + pages - 1) / pages), kSelThreads,
                                 bytes, s>>>(a, tile_rows, pages);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      const dim3 all(a.row_n, a.Hkv);
      e = heads == 4   ? run_exact<4>(cache_choose64_kernel<4>, all, exact, dev, a, s)
          : heads == 2 ? run_exact<2>(cache_choose64_kernel<2>, all, exact, dev, a, s)
                       : run_exact<1>(cache_choose64_kernel<1>, all, exact, dev, a, s);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_cache_select(const CacheArgs& a, cudaStream_t s) {
  return a.d == 128 ? select_d<128>(a, s) : select_d<64>(a, s);
}

}  // namespace ta
