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
// amax is not finite.
__device__ __forceinline__ float token_scale(float amax) {
  if (amax == 0.0f) return 1.0f;
  if (!(amax < __int_as_float(0x7f800000))) return __int_as_float(0x7fffffff);
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
// n_select - n_first - n_recent pages of greatest sum_g M_gj, in fp64 so that
// the choice depends on the inputs and not on an order of summation.
//
// The logits are fp64 matrix products (mma.sync m8n8k4): a warp holds the
// means of 8 pages as A fragments and runs over the (row, query head) columns
// of its tile.
constexpr int kSelThreads = 256;
constexpr int kSelPages = 128;         // pages of a logits block
constexpr int kSelCols = 64;           // (row, head) columns of a logits block

__device__ __forceinline__ void dmma(double (&c)[2], double a, double b) {
  asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0, %1}, {%2}, {%3}, {%0, %1};"
               : "+d"(c[0]), "+d"(c[1])
               : "d"(a), "d"(b));
}

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

template <int D>
__global__ void __launch_bounds__(kSelThreads) cache_logits_kernel(const CacheArgs a, int tile_rows) {
  extern __shared__ double qs[];
  constexpr int QP = D + 4;            // padded: a column's chunks fall on banks of their own
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tg = lane & 3;
  const int hk = blockIdx.y;
  int s, t0, t1;
  if (a.cu) {
    // tiles of sequence s start at cu[s] / tile_rows + s
    int lo = 0, hi = a.S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (max(a.cu[mid], 0) / tile_rows + mid <= (int)blockIdx.x) lo = mid; else hi = mid - 1;
    }
    s = lo;
    const int c0 = max(a.cu[s], 0);
    t0 = c0 + ((int)blockIdx.x - (c0 / tile_rows + s)) * tile_rows;
    t1 = min(min(a.cu[s + 1], rows_used(a)), t0 + tile_rows);
  } else {
    s = t0 = blockIdx.x;
    t1 = t0 + 1;
  }
  if (t0 >= t1) return;
  const RowPages last = row_pages(a, t1 - 1, s);   // the tile's longest row
  const int j_end = min(last.c1, (int)(blockIdx.z + 1) * kSelPages);
  const int j0 = blockIdx.z * kSelPages;
  if (j0 >= j_end) return;
  const int cols = (t1 - t0) * a.G, tiles = (cols + 7) / 8;
  for (int i = threadIdx.x; i < tiles * 8 * (D / 2); i += kSelThreads) {
    const int c = i / (D / 2), d = 2 * (i - c * (D / 2));
    double2 x = make_double2(0.0, 0.0);
    if (c < cols) {
      const int r = c / a.G, h = hk * a.G + (c - r * a.G);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(a.q + (int64_t)(t0 + r) * a.sq_t + (int64_t)h * a.sq_h + d);
      x = make_double2((double)bf_lo(w), (double)bf_hi(w));
    }
    *reinterpret_cast<double2*>(qs + c * QP + d) = x;
  }
  __syncthreads();
  for (int j = j0 + warp * 8; j < j_end; j += (kSelThreads / 32) * 8) {
    const int page_j = j + g;
    int page = -1;
    if (page_j < j_end) page = page_of(a, s, page_j);
    double am[D / 16][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (page >= 0)
        v = __ldg(reinterpret_cast<const float4*>(a.k_mean + ((int64_t)page * a.Hkv + hk) * D + 16 * i + 4 * tg));
      am[i][0] = v.x, am[i][1] = v.y, am[i][2] = v.z, am[i][3] = v.w;
    }
    for (int ct = 0; ct < tiles; ++ct) {
      double c0[2] = {0.0, 0.0}, c1[2] = {0.0, 0.0};
      const double* q = qs + (ct * 8 + g) * QP + 4 * tg;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const double2 x = *reinterpret_cast<const double2*>(q + 16 * i);
        const double2 y = *reinterpret_cast<const double2*>(q + 16 * i + 2);
        dmma(c0, am[i][0], x.x);
        dmma(c1, am[i][1], x.y);
        dmma(c0, am[i][2], y.x);
        dmma(c1, am[i][3], y.y);
      }
      if (page_j < j_end) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = ct * 8 + 2 * tg + e;
          if (c >= cols) continue;
          const int r = c / a.G, h = hk * a.G + (c - r * a.G);
          a.scratch[((int64_t)(t0 + r) * a.H + h) * a.max_pages + page_j] =
              page < 0 ? -__longlong_as_double(0x7ff0000000000000ll) : (c0[e] + c1[e]) * a.scale;
        }
      }
    }
  }
}

__device__ __forceinline__ double block_max(double x, double* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmax(x, __shfl_xor_sync(0xffffffffu, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < kSelThreads / 32; ++w) x = fmax(x, red[w]);
  return x;
}
__device__ __forceinline__ double block_sum(double x, double* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < kSelThreads / 32; ++w) x += red[w];
  return x;
}

__global__ void __launch_bounds__(kSelThreads) cache_choose_kernel(const CacheArgs a) {
  extern __shared__ double mass[];     // one for each competing page
  __shared__ double red[kSelThreads / 32];
  __shared__ int hist[256];
  __shared__ int found[2];
  __shared__ int wsum[2][kSelThreads / 32];
  const int t = blockIdx.x, hk = blockIdx.y, tid = threadIdx.x;
  if (t >= rows_used(a)) return;
  const int s = row_seq(a, t);
  const RowPages r = row_pages(a, t, s);
  int* sel = a.sel + ((int64_t)t * a.Hkv + hk) * a.n_select;
  const int nc = r.c1 - r.c0;
  if (r.n <= a.n_select) {
    for (int i = tid; i < a.n_select; i += kSelThreads) sel[i] = i < r.n ? i : -1;
    return;
  }
  int want = a.n_select - a.n_first - a.n_recent;   // < nc here

  // ---- masses ----
  for (int j = tid; j < nc; j += kSelThreads) mass[j] = 0.0;
  for (int gq = 0; gq < a.G; ++gq) {
    const double* l = a.scratch + ((int64_t)t * a.H + hk * a.G + gq) * a.max_pages + r.c0;
    double mx = -__longlong_as_double(0x7ff0000000000000ll);
    for (int j = tid; j < nc; j += kSelThreads)
      if (isfinite(l[j])) mx = fmax(mx, l[j]);
    mx = block_max(mx, red);
    if (mx == -__longlong_as_double(0x7ff0000000000000ll)) continue;
    double sum = 0.0;
    for (int j = tid; j < nc; j += kSelThreads)
      if (isfinite(l[j])) sum += exp(l[j] - mx);
    const double inv = 1.0 / block_sum(sum, red);
    for (int j = tid; j < nc; j += kSelThreads)
      if (isfinite(l[j])) mass[j] += exp(l[j] - mx) * inv;
  }
  __syncthreads();

  // ---- the want-th greatest mass: radix select on the bits (masses are not
  // negative, so their bits order as they do), most significant byte first ----
  unsigned long long pivot = 0;        // every kept mass is >= pivot
  int equal = 0;                       // of those equal to it, this many are kept (0: all)
  if (want > 0) {
    unsigned long long mask = 0;
    int need = want;
    for (int shift = 56; shift >= 0; shift -= 8) {
      hist[tid] = 0;
      __syncthreads();
      for (int j = tid; j < nc; j += kSelThreads) {
        const unsigned long long b = (unsigned long long)__double_as_longlong(mass[j]);
        if ((b & mask) == pivot) atomicAdd(&hist[(b >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid < 32) {
        // lane i holds bins 255 - 8 i .. 248 - 8 i
        int c = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) c += hist[255 - 8 * tid - u];
        int inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (tid >= o) inc += y;
        }
        int before = inc - c;
        if (before < need && inc >= need) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int bin = 255 - 8 * tid - u;
            if (before < need && before + hist[bin] >= need) {
              found[0] = bin;
              found[1] = before;
            }
            before += hist[bin];
          }
        }
      }
      __syncthreads();
      const int bin = found[0], in_bin = hist[bin];
      need -= found[1];
      pivot |= (unsigned long long)bin << shift;
      mask |= 255ull << shift;
      __syncthreads();
      if (in_bin == need) {            // the whole bin is kept
        need = 0;
        break;
      }
    }
    equal = need;
  }

  // ---- the list, in page order ----
  int at = 0, eq_seen = 0;
  for (int base = 0; base < r.n; base += kSelThreads) {
    const int j = base + tid;
    bool keep = j < r.c0 || (j >= r.c1 && j < r.n), eq = false;
    if (j >= r.c0 && j < r.c1 && want > 0) {
      const unsigned long long b = (unsigned long long)__double_as_longlong(mass[j - r.c0]);
      if (equal == 0) {
        keep = b >= pivot;
      } else {
        keep = b > pivot;
        eq = b == pivot;
      }
    }
    const uint32_t be = __ballot_sync(0xffffffffu, eq), below = (1u << (tid & 31)) - 1;
    if ((tid & 31) == 0) wsum[0][tid >> 5] = __popc(be);
    __syncthreads();
    int e0 = eq_seen, e_all = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < (tid >> 5)) e0 += wsum[0][w];
      e_all += wsum[0][w];
    }
    if (eq) keep = e0 + __popc(be & below) < equal;
    eq_seen += e_all;
    const uint32_t bk = __ballot_sync(0xffffffffu, keep);
    if ((tid & 31) == 0) wsum[1][tid >> 5] = __popc(bk);
    __syncthreads();
    int k0 = at, k_all = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < (tid >> 5)) k0 += wsum[1][w];
      k_all += wsum[1][w];
    }
    if (keep) {
      const int i = k0 + __popc(bk & below);
      if (i < a.n_select) sel[i] = j;
    }
    at += k_all;
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

cudaError_t launch_cache_select(const CacheArgs& a, cudaStream_t s) {
  const int tile_rows = a.cu ? (a.G >= kSelCols ? 1 : kSelCols / a.G) : 1;
  const int64_t tiles = a.cu ? (int64_t)(a.T / tile_rows) + a.S : a.S;
  const int cols = (tile_rows * a.G + 7) / 8 * 8;
  const int bytes = cols * (a.d + 4) * 8;
  const dim3 grid((unsigned)tiles, a.Hkv, (a.max_pages + kSelPages - 1) / kSelPages);
  auto go = [&](auto kernel) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kSelThreads, bytes, s>>>(a, tile_rows);
    return cudaGetLastError();
  };
  cudaError_t e = a.d == 128 ? go(cache_logits_kernel<128>) : go(cache_logits_kernel<64>);
  if (e != cudaSuccess) return e;
  const int mb = a.max_pages * 8;
  e = cudaFuncSetAttribute(cache_choose_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, mb);
  if (e != cudaSuccess) return e;
  cache_choose_kernel<<<dim3(a.T, a.Hkv), kSelThreads, mb, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ta
