// ta_cache_attn.cu -- attention of single rows over a paged key-value cache:
// one new token of each sequence over all of its keys (decode), or every row
// over the pages of its own list (sparse).
//
// Mathematics, per row and query head: with s_i = scale * q . k_i over the
// row's visible keys i, m = max s_i, O = sum_i 2^{(s_i - m) log2 e} v_i / l and
// l = sum_i 2^{(s_i - m) log2 e}, folded in one pass with a running maximum.
// Parts of a row with maxima m_a, sums l_a and numerators n_a join as
// m = max m_a, l = sum 2^{m_a - m} l_a, n = sum 2^{m_a - m} n_a.
//
// Layout of the work.  An item is a (row, key head); its keys go in units of
// 128.  The units of all items, in order, are cut into equal runs, one for
// each CTA, whatever the lengths: a run may end inside an item, whose parts
// then meet in the workspace, where the CTA that arrives last joins them in
// the order of the parts.  Within a CTA one warp loads (TMA, one box a page
// and 128-byte column) and four warps compute, each on 32 keys of a unit with
// a softmax state of its own, joined at the item's end.
//
// The products run transposed, S^T = K Q^T and O^T = V^T P^T, with mma.sync
// m16n8k16: the keys (or the head dim) fill the 16 rows and the query heads
// that share a key head the 8 columns, so a group of up to 8 heads wastes
// nothing of the M side.  The operator is bound by the cache's bytes: a key
// head's 256 bytes of one key need 2 * 8 * 128 multiply-adds at most, a tenth
// of what mma.sync does in that time, so tcgen05 (M = 128 rows) would only
// idle.  P is rounded to bf16 for the second product (at most 2^-9 relative
// for each weight, the size of O's own rounding); l sums the unrounded
// weights in fp32.
#include "ta_cache.cuh"

namespace ta {
namespace {

constexpr int kUnit = 128;               // keys of a unit (one pipeline stage)
constexpr int kWarps = 4;                // computing warps, 32 keys of a unit each
constexpr int kThreads = 32 * (kWarps + 1);

template <int D, bool FP8, int NT>
struct Cfg {
  static constexpr int kRow = D * (FP8 ? 1 : 2);          // bytes of a key
  static constexpr int kCols = kRow > 128 ? 2 : 1;        // 128-byte columns of a row
  static constexpr int kColB = kRow / kCols;              // 128 or 64
  static constexpr int kTile = kUnit * kRow;
  static constexpr int kScales = FP8 ? kUnit * 4 : 0;
  static constexpr int kStage = 2 * kTile + 2 * kScales;
  static constexpr int kStages = kStage > 40000 ? 3 : (kStage > 20000 ? 5 : 8);
  static constexpr int kRegs = D / 16 * NT * 4;           // accumulators of a lane
  static constexpr int oJoin = kStages * ((kStage + 1023) / 1024 * 1024);
  static constexpr int oML = oJoin + 2 * kRegs * 32 * 4;
  static constexpr int oCnt = oML + 2 * 2 * kWarps * kMaxTileHeads * 4;  // m, l; items take turns
  static constexpr int oBar = oCnt + kStages * 8 * 4;
  static constexpr int oMisc = oBar + 2 * kStages * 8;
  static constexpr int oPre = oMisc + 64;
  static constexpr int kBytes = oPre + 1024;              // 1024 to align; + a decode's prefix
  static constexpr int kStageStep = (kStage + 1023) / 1024 * 1024;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
// Two e4m3 codes, in bytes 1 and 3 of w, to bf16x2 (exact): exponent and
// mantissa moved to bf16's places give the value times 2^-120 (the biases
// differ by 120; a subnormal code becomes a bf16 subnormal), which the
// product with 2^120 undoes.  The NaN code comes out as 480: a token that
// holds one has a NaN scale.
__device__ __forceinline__ uint32_t e4m3_bf16x2(uint32_t w) {
  const uint32_t t = ((w >> 4) & 0x07F007F0u) | (w & 0x80008000u);
  uint32_t r;
  asm("mul.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(t), "r"(0x7B807B80u));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}

// Where a run of units stands: row, head group, and unit of that item.
template <bool SPARSE>
struct Cursor {
  int row, hx, k, units;
  __device__ __forceinline__ int units_of(const CacheArgs& a, const int* pre, int r) const {
    return SPARSE ? (a.n_select * a.page_size + kUnit - 1) / kUnit : pre[r + 1] - pre[r];
  }
  __device__ __forceinline__ void start(const CacheArgs& a, const int* pre, int rows, int HX,
                                        int64_t u) {
    if (SPARSE) {
      units = units_of(a, pre, 0);
      row = (int)(u / ((int64_t)units * HX));
      const int r = (int)(u - (int64_t)row * units * HX);
      hx = r / units;
      k = r - hx * units;
    } else {
      int lo = 0, hi = rows - 1;      // last row whose base is not above u (it has units)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)pre[mid] * HX <= u) lo = mid; else hi = mid - 1;
      }
      row = lo;
      units = units_of(a, pre, row);
      const int r = (int)(u - (int64_t)pre[row] * HX);
      hx = r / units;
      k = r - hx * units;
    }
  }
  // To the next unit; only while one follows.
  __device__ __forceinline__ void next(const CacheArgs& a, const int* pre, int HX) {
    if (++k < units) return;
    k = 0;
    if (++hx < HX) return;
    hx = 0;
    do {
      ++row;
      units = units_of(a, pre, row);
    } while (units == 0);
  }
};

template <int D, bool FP8, int NT, bool SPARSE>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                      const CacheArgs a) {
  using C = Cfg<D, FP8, NT>;
  constexpr int NH = 8 * NT;                       // query heads of an item
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* cnt = reinterpret_cast<int*>(smem + C::oCnt);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::oBar);
  uint64_t* empty = full + C::kStages;
  int* misc = reinterpret_cast<int*>(smem + C::oMisc);
  int* pre = reinterpret_cast<int*>(smem + C::oPre);
  float* const sm_m0 = reinterpret_cast<float*>(smem + C::oML);
  const AbortCtx abort{misc, a.status};

  const int HG = (a.G + NH - 1) / NH;              // items of one key head
  const int HX = a.Hkv * HG;
  const int rows = SPARSE ? rows_used(a) : a.S;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    misc[0] = 0;
    fence_mbar_init();
  }

  // ---- units of all items ----
  int64_t W;
  if (SPARSE) {
    W = (int64_t)rows * HX * ((a.n_select * a.page_size + kUnit - 1) / kUnit);
  } else {
    // pre[r] = units of one head over rows before r
    const int per = (rows + kThreads - 1) / kThreads;
    const int r0 = min(rows, tid * per), r1 = min(rows, r0 + per);
    int sum = 0;
    for (int r = r0; r < r1; ++r) sum += (seq_len(a, r) + kUnit - 1) / kUnit;
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) misc[4 + warp] = inc;
    __syncthreads();
    int base = inc - sum;
    for (int w = 0; w < warp; ++w) base += misc[4 + w];
    for (int r = r0; r < r1; ++r) {
      pre[r] = base;
      base += (seq_len(a, r) + kUnit - 1) / kUnit;
    }
    if (tid == kThreads - 1) pre[rows] = base;
    __syncthreads();
    W = (int64_t)pre[rows] * HX;
    // empty sequences have no unit: their rows are written here
    for (int r = blockIdx.x; r < rows; r += gridDim.x) {
      if (pre[r + 1] != pre[r]) continue;
      for (int i = tid; i < a.H * D; i += kThreads) {
        const int h = i / D;
        a.o[(int64_t)r * a.so_t + (int64_t)h * a.so_h + (i - h * D)] = __float2bfloat16_rn(0.0f);
      }
      if (a.lse)
        for (int h = tid; h < a.H; h += kThreads)
          a.lse[(int64_t)r * a.H + h] = -__int_as_float(0x7f800000);
    }
  }
  __syncthreads();
  const int64_t n = W < (int64_t)gridDim.x ? W : (int64_t)gridDim.x;
  if ((int64_t)blockIdx.x >= n) return;
  const int64_t u0 = W * blockIdx.x / n, u1 = W * (blockIdx.x + 1) / n;
  const int n_units = (int)(u1 - u0);
  Cursor<SPARSE> cur;
  cur.start(a, pre, rows, HX, u0);

  if (warp == kWarps) {
    // ---- loads: lane i brings page i of the unit ----
    const int ppu = kUnit >> a.ps_log2;
    int row = -1, s = 0, len = 0;
    int issued = 0;
    for (int i = 0; i < n_units; ++i) {
      const int st = i % C::kStages;
      if (cur.row != row) {
        row = cur.row;
        s = SPARSE ? row_seq(a, row) : row;
        len = SPARSE ? row_pos(a, row, s) + 1 : seq_len(a, s);
      }
      const int hk = cur.hx / HG;
      int page = 0, vc = 0;
      if (lane < ppu) {
        int e = cur.k * ppu + lane;
        if (SPARSE) e = e < a.n_select ? a.sel[((int64_t)row * a.Hkv + hk) * a.n_select + e] : -1;
        if (e >= 0 && e < a.max_pages) vc = min(a.page_size, max(0, len - (e << a.ps_log2)));
        if (vc > 0) {
          page = page_of(a, s, e);
          if (page < 0) vc = 0;
        }
      }
      const uint32_t live = __ballot_sync(0xffffffffu, vc > 0);
      if (i >= C::kStages && !mbar_wait(&empty[st], ((i / C::kStages) - 1) & 1, abort, 1)) break;
      unsigned char* stage = smem + st * C::kStageStep;
      const int v16 = __shfl_sync(0xffffffffu, vc, (lane & 7) >> (a.ps_log2 - 4));
      if (lane < 8)
        cnt[st * 8 + lane] = min(16, max(0, v16 - 16 * (lane & ((1 << (a.ps_log2 - 4)) - 1))));
      __syncwarp();
      if (lane == 0) {
        const uint32_t bytes = (uint32_t)a.page_size * (2 * C::kRow + (FP8 ? 8 : 0));
        mbar_arrive_expect_tx(&full[st], bytes * __popc(live));
      }
      __syncwarp();
      if (vc > 0) {
        const int off = lane << a.ps_log2;         // first key of the page in the unit
#pragma unroll
        for (int c = 0; c < C::kCols; ++c) {
          unsigned char* dst = stage + c * (kUnit * C::kColB) + off * C::kColB;
          tma_load_4d(dst, &mk, &full[st], c * 64, 0, hk, page);
          tma_load_4d(dst + C::kTile, &mv, &full[st], c * 64, 0, hk, page);
        }
        if (FP8) {
          const int64_t so = ((int64_t)page * a.Hkv + hk) << a.ps_log2;
          bulk_load(stage + 2 * C::kTile + off * 4, a.k_scale + so, a.page_size * 4, &full[st]);
          bulk_load(stage + 2 * C::kTile + C::kScales + off * 4, a.v_scale + so, a.page_size * 4,
                    &full[st]);
        }
      }
      issued = i + 1;
      if (i + 1 < n_units) cur.next(a, pre, HX);
    }
    if (*abort.abort) {
      // nothing may still be writing shared memory when the CTA ends
      for (int i = max(0, issued - C::kStages); i < issued; ++i)
        mbar_wait_drain(&full[i % C::kStages], (i / C::kStages) & 1);
    }
    return;
  }

  // ---- compute ----
  const int g = lane >> 2, tg = lane & 3;
  const float sc = a.scale_log2;
  uint32_t qf[D / 16][NT][2];
  float acc[D / 16][NT][4];
  float m[NT][2], l[NT][2];
  float* join = reinterpret_cast<float*>(smem + C::oJoin);
  const float kNegInf = -__int_as_float(0x7f800000);
  bool fresh = true;                               // no unit of the item taken yet
  int k_first = 0;                                 // first unit of the item in this run
  int turn = 0;
  float* sm_m = sm_m0;

  for (int i = 0; i < n_units; ++i) {
    const int st = i % C::kStages;
    const int hk = cur.hx / HG, h0 = hk * a.G + (cur.hx - hk * HG) * NH;
    const int nh = min(NH, (hk + 1) * a.G - h0);   // heads in use
    if (fresh) {
      fresh = false;
      k_first = cur.k;
      const __nv_bfloat16* q = a.q + (int64_t)cur.row * a.sq_t + (int64_t)h0 * a.sq_h;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bool on = nt * 8 + g < nh;
        const __nv_bfloat16* qh = q + (int64_t)(nt * 8 + g) * a.sq_h;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          // bf16 keys: k index of the fragment = head element; FP8: a lane's
          // four k indices are four consecutive elements (as its keys load)
          const int d0 = c * 16 + (FP8 ? 4 * tg : 2 * tg), d1 = d0 + (FP8 ? 2 : 8);
          qf[c][nt][0] = on ? *reinterpret_cast<const uint32_t*>(qh + d0) : 0u;
          qf[c][nt][1] = on ? *reinterpret_cast<const uint32_t*>(qh + d1) : 0u;
        }
        m[nt][0] = m[nt][1] = kNegInf;
        l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[c][nt][j] = 0.0f;
      }
    }
    const bool ok = mbar_wait(&full[st], (i / C::kStages) & 1, abort, 2);
    const int c0 = ok ? cnt[st * 8 + 2 * warp] : 0, c1 = ok ? cnt[st * 8 + 2 * warp + 1] : 0;
    if (c0 | c1) {
      const uint32_t kbase = smem_u32(smem + st * C::kStageStep);
      const uint32_t vbase = kbase + C::kTile;
      const int key0 = warp * 32;
      float s[2][NT][4];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[kt][nt][j] = 0.0f;
      // address of 16-byte chunk c of key r (swizzled as TMA stored it)
      auto chunk = [&](uint32_t base, int r, int c) -> uint32_t {
        if constexpr (C::kColB == 128)
          return base + (c >> 3) * (kUnit * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        else
          return base + r * 64 + (((c & 3) ^ ((r >> 1) & 3)) << 4);
      };
      if constexpr (!FP8) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            uint32_t r[4];
            ldsm4(r, chunk(kbase, key0 + kt * 16 + (lane & 15), 2 * c + (lane >> 4)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816(s[kt][nt], r[0], r[1], r[2], r[3], qf[c][nt][0], qf[c][nt][1]);
          }
      } else {
#pragma unroll
        for (int c = 0; c < D / 16; c += 2)
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            uint32_t r[4];   // rows 0-7 and 8-15 of chunk c, then of chunk c + 1
            ldsm4(r, chunk(kbase, key0 + kt * 16 + (lane & 15), c + (lane >> 4)));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t x = r[2 * e], y = r[2 * e + 1];
              const uint32_t a0 = e4m3_bf16x2(__byte_perm(x, 0, 0x1404));
              const uint32_t a2 = e4m3_bf16x2(__byte_perm(x, 0, 0x3424));
              const uint32_t a1 = e4m3_bf16x2(__byte_perm(y, 0, 0x1404));
              const uint32_t a3 = e4m3_bf16x2(__byte_perm(y, 0, 0x3424));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(s[kt][nt], a0, a1, a2, a3, qf[c + e][nt][0], qf[c + e][nt][1]);
            }
          }
      }
      // hidden keys, key scales, running maximum
      const float* kss = reinterpret_cast<const float*>(smem + st * C::kStageStep + 2 * C::kTile);
      const float* vss = kss + kUnit;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = kNegInf;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        const int c = kt ? c1 : c0;
        float f0 = 1.0f, f1 = 1.0f;
        if (FP8) {
          f0 = kss[key0 + kt * 16 + g];
          f1 = kss[key0 + kt * 16 + g + 8];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            s[kt][nt][j] = g < c ? (FP8 ? s[kt][nt][j] * f0 : s[kt][nt][j]) : kNegInf;
            s[kt][nt][j + 2] = g + 8 < c ? (FP8 ? s[kt][nt][j + 2] * f1 : s[kt][nt][j + 2]) : kNegInf;
            mx[nt][j] = fmax3(mx[nt][j], s[kt][nt][j], s[kt][nt][j + 2]);
          }
      }
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            mx[nt][j] = fmaxf(mx[nt][j], __shfl_xor_sync(0xffffffffu, mx[nt][j], o));
          mx[nt][j] = fmaxf(mx[nt][j], m[nt][j]);
          up |= mx[nt][j] > m[nt][j];
        }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float f = m[nt][j] == kNegInf ? 0.0f : ex2((m[nt][j] - mx[nt][j]) * sc);
            m[nt][j] = mx[nt][j];
            l[nt][j] *= f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              acc[c][nt][j] *= f;
              acc[c][nt][j + 2] *= f;
            }
          }
      }
      // weights, their sums, and P^T as the second product's B operand
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mm[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) mm[j] = m[nt][j] == kNegInf ? 0.0f : m[nt][j] * sc;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          const int c = kt ? c1 : c0;
          float p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p[j] = ex2(fmaf(s[kt][nt][j], sc, -mm[j & 1]));
            l[nt][j & 1] += p[j];
          }
          if (FP8) {
            const float f0 = g < c ? vss[key0 + kt * 16 + g] : 0.0f;
            const float f1 = g + 8 < c ? vss[key0 + kt * 16 + g + 8] : 0.0f;
            p[0] *= f0;
            p[1] *= f0;
            p[2] *= f1;
            p[3] *= f1;
          }
          pf[kt][nt][0] = movm(pack_bf16(p[0], p[1]));
          pf[kt][nt][1] = movm(pack_bf16(p[2], p[3]));
        }
      }
      // O^T += V^T P^T; slots behind the last key hold anything, NaN included
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        const int c = kt ? c1 : c0;
        if (c == 0) continue;
        const uint32_t m0 = (2 * tg < c ? 0xFFFFu : 0u) | (2 * tg + 1 < c ? 0xFFFF0000u : 0u);
        const uint32_t m1 = (2 * tg + 8 < c ? 0xFFFFu : 0u) | (2 * tg + 9 < c ? 0xFFFF0000u : 0u);
        if constexpr (!FP8) {
#pragma unroll
          for (int cd = 0; cd < D / 16; ++cd) {
            uint32_t r[4];   // keys 0-7 by d 0-7 and 8-15, then keys 8-15
            ldsm4t(r, chunk(vbase, key0 + kt * 16 + (lane & 7) + ((lane >> 4) << 3),
                            2 * cd + ((lane >> 3) & 1)));
            r[0] &= m0;
            r[1] &= m0;
            r[2] &= m1;
            r[3] &= m1;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816(acc[cd][nt], r[0], r[1], r[2], r[3], pf[kt][nt][0], pf[kt][nt][1]);
          }
        } else {
#pragma unroll
          for (int cd = 0; cd < D / 16; cd += 2) {
            uint32_t r[4];   // chunk cd by keys 0-7 and 8-15, then chunk cd + 1
            ldsm4t(r, chunk(vbase, key0 + kt * 16 + (lane & 15), cd + (lane >> 4)));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t x = r[2 * e], y = r[2 * e + 1];
              const uint32_t a0 = e4m3_bf16x2(__byte_perm(x, 0, 0x2404)) & m0;
              const uint32_t a1 = e4m3_bf16x2(__byte_perm(x, 0, 0x3414)) & m0;
              const uint32_t a2 = e4m3_bf16x2(__byte_perm(y, 0, 0x2404)) & m1;
              const uint32_t a3 = e4m3_bf16x2(__byte_perm(y, 0, 0x3414)) & m1;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(acc[cd + e][nt], a0, a1, a2, a3, pf[kt][nt][0], pf[kt][nt][1]);
            }
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);

    if (cur.k + 1 == cur.units || i + 1 == n_units) {
      // ---- join the four warps ----
      // (the state of an item may still be read while the next one is written)
      float* sm_l = sm_m + kWarps * kMaxTileHeads;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], o);
          if (g == 0) {
            sm_m[warp * kMaxTileHeads + nt * 8 + 2 * tg + j] = m[nt][j];
            sm_l[warp * kMaxTileHeads + nt * 8 + 2 * tg + j] = l[nt][j];
          }
        }
      compute_sync();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float mm = kNegInf;
          for (int w = 0; w < kWarps; ++w)
            mm = fmaxf(mm, sm_m[w * kMaxTileHeads + nt * 8 + 2 * tg + j]);
          const float f = m[nt][j] == kNegInf ? 0.0f : ex2((m[nt][j] - mm) * sc);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            acc[c][nt][j] *= f;
            acc[c][nt][j + 2] *= f;
          }
        }
      float* mine = join + (warp & 1) * (C::kRegs * 32) + lane;
      if (warp >= 2) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) mine[((c * NT + nt) * 4 + j) * 32] = acc[c][nt][j];
      }
      compute_sync();
      if (warp < 2) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) mine[((c * NT + nt) * 4 + j) * 32] += acc[c][nt][j];
      }
      compute_sync();
      // element (head n, pair of d) of the joined numerators
      auto joined = [&](int nn, int d) -> float {
        const int dd = d & 15;
        const int gg = FP8 ? dd >> 1 : dd & 7, hi = FP8 ? dd & 1 : dd >> 3;
        const int at = (((d >> 4) * NT + (nn >> 3)) * 4 + hi * 2 + (nn & 1)) * 32 + gg * 4 + ((nn & 7) >> 1);
        return join[at] + join[C::kRegs * 32 + at];
      };
      auto state = [&](int nn, float& mm, float& ll) {
        mm = kNegInf;
        ll = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w * kMaxTileHeads + nn]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = sm_m[w * kMaxTileHeads + nn];
          ll += mw == kNegInf ? 0.0f : ex2((mw - mm) * sc) * sm_l[w * kMaxTileHeads + nn];
        }
      };
      __nv_bfloat16* out = a.o + (int64_t)cur.row * a.so_t + (int64_t)h0 * a.so_h;
      auto put = [&](int nn, int d, float x, float y, float mm, float ll) {
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        *reinterpret_cast<uint32_t*>(out + (int64_t)nn * a.so_h + d) = pack_bf16(x * inv, y * inv);
        if (d == 0 && a.lse)
          a.lse[(int64_t)cur.row * a.H + h0 + nn] =
              ll == 0.0f ? kNegInf : (mm * sc + log2f(ll)) * 0.6931471805599453f;
      };
      const bool begins = k_first == 0, ends = cur.k + 1 == cur.units;
      if (begins && ends) {
        for (int e = tid; e < nh * (D / 2); e += 32 * kWarps) {
          const int nn = e / (D / 2), d = 2 * (e - nn * (D / 2));
          float mm, ll;
          state(nn, mm, ll);
          put(nn, d, joined(nn, d), joined(nn, d + 1), mm, ll);
        }
      } else {
        // a part: the item's first part stands in slot 1 of its CTA, the
        // others in slot 0 of theirs
        const int64_t b0 = u0 + i - cur.k;                 // the item's first unit
        const int64_t b1 = b0 + cur.units - 1;             // and its last
        const int cf = (int)(((b0 + 1) * n - 1) / W), cl = (int)(((b1 + 1) * n - 1) / W);
        const int slot = 2 * (int)blockIdx.x + (begins ? 1 : 0);
        float* po = a.part_o + (int64_t)slot * (kMaxTileHeads * 128);
        float* pml = a.part_ml + slot * (2 * kMaxTileHeads);
        for (int e = tid; e < nh * (D / 2); e += 32 * kWarps) {
          const int nn = e / (D / 2), d = 2 * (e - nn * (D / 2));
          __stcg(reinterpret_cast<float2*>(po + nn * D + d), make_float2(joined(nn, d), joined(nn, d + 1)));
          if (d == 0) {
            float mm, ll;
            state(nn, mm, ll);
            __stcg(pml + nn, mm);
            __stcg(pml + kMaxTileHeads + nn, ll);
          }
        }
        __threadfence();
        compute_sync();
        if (tid == 0)
          misc[1] = atomicInc(reinterpret_cast<unsigned int*>(a.counters) + cf, (unsigned)(cl - cf)) ==
                    (unsigned)(cl - cf);
        compute_sync();
        if (misc[1]) {
          __threadfence();
          for (int e = tid; e < nh * (D / 2); e += 32 * kWarps) {
            const int nn = e / (D / 2), d = 2 * (e - nn * (D / 2));
            float mm = kNegInf, ll = 0.0f, x = 0.0f, y = 0.0f;
            for (int c = cf; c <= cl; ++c)
              mm = fmaxf(mm, __ldcg(a.part_ml + (2 * c + (c == cf)) * (2 * kMaxTileHeads) + nn));
            for (int c = cf; c <= cl; ++c) {
              const int sl = 2 * c + (c == cf);
              const float mw = __ldcg(a.part_ml + sl * (2 * kMaxTileHeads) + nn);
              const float f = mw == kNegInf ? 0.0f : ex2((mw - mm) * sc);
              const float2 v = __ldcg(reinterpret_cast<const float2*>(
                  a.part_o + (int64_t)sl * (kMaxTileHeads * 128) + nn * D + d));
              ll += f * __ldcg(a.part_ml + sl * (2 * kMaxTileHeads) + kMaxTileHeads + nn);
              x += f * v.x;
              y += f * v.y;
            }
            put(nn, d, x, y, mm, ll);
          }
        }
      }
      fresh = true;
      turn ^= 1;
      sm_m = sm_m0 + turn * (2 * kWarps * kMaxTileHeads);
    }
    if (i + 1 < n_units) cur.next(a, pre, HX);
  }
}

template <int D, bool FP8, int NT, bool SPARSE>
cudaError_t run(const CacheArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  using C = Cfg<D, FP8, NT>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int bytes = C::kBytes + (SPARSE ? 0 : (a.S + 1) * 4);
  auto k = cache_attn_kernel<D, FP8, NT, SPARSE>;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  // no more CTAs than units the call can have
  const int64_t HX = (int64_t)a.Hkv * ((a.G + 8 * NT - 1) / (8 * NT));
  const int64_t per = ((int64_t)(SPARSE ? a.n_select : a.max_pages) * a.page_size + kUnit - 1) / kUnit;
  int64_t grid = (SPARSE ? a.T : a.S) * HX * per;
  if (grid > sms) grid = sms;
  if (grid > kMaxAttnCtas) grid = kMaxAttnCtas;
  k<<<(int)grid, kThreads, bytes, s>>>(mk, mv, a);
  return cudaGetLastError();
}

template <int D, bool FP8>
cudaError_t pick(const CacheArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, bool sparse,
                 cudaStream_t s) {
  // groups of more than 8 query heads take two column tiles, so that each key
  // is read once for up to 16 of them
  if (a.G <= 8)
    return sparse ? run<D, FP8, 1, true>(a, mk, mv, s) : run<D, FP8, 1, false>(a, mk, mv, s);
  return sparse ? run<D, FP8, 2, true>(a, mk, mv, s) : run<D, FP8, 2, false>(a, mk, mv, s);
}

}  // namespace

cudaError_t launch_cache_attn(const CacheArgs& a, const CUtensorMap& mk, const CUtensorMap& mv,
                              bool sparse, cudaStream_t s) {
  if (a.d == 128)
    return a.fp8 ? pick<128, true>(a, mk, mv, sparse, s) : pick<128, false>(a, mk, mv, sparse, s);
  return a.fp8 ? pick<64, true>(a, mk, mv, sparse, s) : pick<64, false>(a, mk, mv, sparse, s);
}

}  // namespace ta
