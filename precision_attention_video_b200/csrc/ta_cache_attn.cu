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
// 128 (bf16, d = 128) or 256.  The units of all items, in order, are cut into
// equal runs, one for each CTA, whatever the lengths: a run may end inside an
// item, whose parts then meet in the workspace, where the CTA that arrives
// last joins them in the order of the parts.  Within a CTA one warp loads
// (TMA, one box a page and 128-byte column) and eight warps compute, each on
// 16 or 32 keys of a unit with a softmax state of its own, joined at the
// item's end.  (Four warps instead of eight: 238 us against 133 for 4
// sequences of up to 131072 tokens in FP8, with the conversions below; one
// warp on a scheduler does not hide its own latencies.)
//
// The products run transposed, S^T = K Q^T and O^T = V^T P^T, with mma.sync
// m16n8k16: the keys (or the head dim) fill the 16 rows and the query heads
// that share a key head the 8 columns, so a group of up to 8 heads wastes
// nothing of the M side.  The operator is bound by the cache's bytes: a key
// head's 256 bytes of one key need 2 * 8 * 128 multiply-adds at most, a tenth
// of what mma.sync does in that time, so tcgen05 (M = 128 rows) would only
// idle.
//
// bf16 caches multiply in bf16, P rounded to it (at most 2^-8 relative for
// each weight, as O's own rounding).  FP8 caches multiply in f16, which holds
// every e4m3 value and which one conversion instruction reaches for two codes
// (bf16 took five on the integer pipe, half of all issue slots); K's scale
// multiplies a score, V's the weight.  l sums the unrounded weights in fp32.
#include <type_traits>

#include "ta_cache.cuh"

namespace ta {
namespace {

template <int D, bool FP8, int NT>
struct Cfg {
  static constexpr int kRow = D * (FP8 ? 1 : 2);          // bytes of a key
  static constexpr int kKT = kRow > 128 ? 1 : 2;          // 16-key tiles of a warp
  static constexpr int kWarps = 8;                        // computing warps, one more loads
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kUnit = kWarps * 16 * kKT;         // keys of a unit (one stage)
  static constexpr int kCols = kRow > 128 ? 2 : 1;        // 128-byte columns of a row
  static constexpr int kColB = kRow / kCols;              // 128 or 64
  static constexpr int kTile = kUnit * kRow;               // 16 or 32 KB
  static constexpr int kScales = FP8 ? kUnit * 4 : 0;
  static constexpr int kStage = 2 * kTile + 2 * kScales;
  static constexpr int kStages = kStage > 40000 ? 3 : 6;
  static constexpr int kRegs = D / 16 * NT * 4;           // accumulators of a lane
  static constexpr int oJoin = kStages * ((kStage + 1023) / 1024 * 1024);
  static constexpr int kJoin = NT == 1 ? 4 : 2;           // warps that join at a time
  static constexpr int oML = oJoin + kJoin * kRegs * 32 * 4;
  static constexpr int oCnt = oML + 2 * 2 * kWarps * 8 * NT * 4;         // m, l; items take turns
  static constexpr int oBar = oCnt + kStages * (kUnit / 16) * 4;
  static constexpr int oMisc = oBar + 2 * kStages * 8;
  static constexpr int oPre = oMisc + 128;
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
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
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
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
// The e4m3 codes in the low or high half of w to f16x2 (exact).
__device__ __forceinline__ uint32_t e4m3_f16x2_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_f16x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
// 2^floor(log2 x) of a normal x > 0.
__device__ __forceinline__ float pow2_of(float x) {
  return __uint_as_float(__float_as_uint(x) & 0x7F800000u);
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
template <int WARPS>
__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory");
}

// Where a run of units stands: row, head group, and unit of that item.
template <bool SPARSE, int UNIT>
struct Cursor {
  int row, hx, k, units;
  __device__ __forceinline__ int units_of(const CacheArgs& a, const int* pre, int r) const {
    return SPARSE ? (a.n_select * a.page_size + UNIT - 1) / UNIT : pre[r + 1] - pre[r];
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

// The softmax state of a warp: 8 NT columns (query heads), D numerators each.
template <int D, int NT>
struct Fold {
  uint32_t qf[D / 16][NT][2];    // the queries, as B fragments
  float acc[D / 16][NT][4];
  float m[NT][2], l[NT][2];      // running maximum (of s * sq, log2 units) and sum
  float sq[NT][2];               // what a raw product counts for, in log2 units
  float vmax;                    // FP8: the numerators' unit, the largest V scale so far
};

// Column nt * 8 + g's query into the fragments (`on`: the column is in use),
// and the state of an item without keys.
template <int D, bool FP8, int NT>
__device__ __forceinline__ void fold_query(Fold<D, NT>& f, int nt, const __nv_bfloat16* qh, bool on, float sc) {
  const int lane = threadIdx.x & 31, tg = lane & 3;
  auto& qf = f.qf;
  auto& sq = f.sq;
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    // bf16 keys: k index of the fragment = head element; FP8: a lane's
    // four k indices are four consecutive elements (as its keys load)
    const int d0 = c * 16 + (FP8 ? 4 * tg : 2 * tg), d1 = d0 + (FP8 ? 2 : 8);
    qf[c][nt][0] = on ? *reinterpret_cast<const uint32_t*>(qh + d0) : 0u;
    qf[c][nt][1] = on ? *reinterpret_cast<const uint32_t*>(qh + d1) : 0u;
  }
  if constexpr (FP8) {
    // FP8 keys are f16 operands, so the query is one too, its largest
    // element scaled to [2^8, 2^9) by a power of two: what falls below
    // f16's smallest step is under 2^-33 of that element
    uint32_t am = 0;
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        am = max(am, max((qf[c][nt][e] & 0x7FFFu) << 16, qf[c][nt][e] & 0x7FFF0000u));
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
    // (a head of zeros or with values that are not finite is left as it is)
    const float ax = __uint_as_float(am);
    const bool plain = ax >= 1e-35f && ax <= 3.4e38f;
    const float up = plain ? 256.0f / pow2_of(ax) : 1.0f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t w = qf[c][nt][e];
        qf[c][nt][e] = pack_f16(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
      }
    const float down = plain ? pow2_of(ax) * 0.00390625f : 1.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j)                // from the lanes that hold head 2 tg + j
      sq[nt][j] = sc * __shfl_sync(0xffffffffu, down, (2 * tg + j) * 4);
  } else {
    sq[nt][0] = sq[nt][1] = sc;
  }
  f.m[nt][0] = f.m[nt][1] = -__int_as_float(0x7f800000);
  f.l[nt][0] = f.l[nt][1] = 0.0f;
#pragma unroll
  for (int c = 0; c < D / 16; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) f.acc[c][nt][j] = 0.0f;
}

// Folds a warp's 16 KT keys (from key0 of the stage on) into its state.
// cn[kt]: keys of tile kt that exist; seen(kt, e, nt, j): whether key g + 8 e
// of it is visible to column nt * 8 + 2 tg + j.
template <class C, int D, bool FP8, int NT, typename Seen>
__device__ __forceinline__ void fold_unit(Fold<D, NT>& f, const unsigned char* stage, int key0,
                                          const int (&cn)[C::kKT], Seen seen) {
  constexpr int KT = C::kKT, kUnit = C::kUnit;
  const int lane = threadIdx.x & 31, g = lane >> 2, tg = lane & 3;
  const float kNegInf = -__int_as_float(0x7f800000);
  auto& qf = f.qf;
  auto& acc = f.acc;
  auto& m = f.m;
  auto& l = f.l;
  auto& sq = f.sq;
  auto& vmax = f.vmax;
  const uint32_t kbase = smem_u32(stage);
  const uint32_t vbase = kbase + C::kTile;
  float s[KT][NT][4];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
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
      for (int kt = 0; kt < KT; ++kt) {
        uint32_t r[4];
        ldsm4(r, chunk(kbase, key0 + kt * 16 + (lane & 15), 2 * c + (lane >> 4)));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816<false>(s[kt][nt], r[0], r[1], r[2], r[3], qf[c][nt][0], qf[c][nt][1]);
      }
  } else {
#pragma unroll
    for (int c = 0; c < D / 16; c += 2)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        uint32_t r[4];   // rows 0-7 and 8-15 of chunk c, then of chunk c + 1
        ldsm4(r, chunk(kbase, key0 + kt * 16 + (lane & 15), c + (lane >> 4)));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t x = r[2 * e], y = r[2 * e + 1];
          const uint32_t a0 = e4m3_f16x2_lo(x), a2 = e4m3_f16x2_hi(x);
          const uint32_t a1 = e4m3_f16x2_lo(y), a3 = e4m3_f16x2_hi(y);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816<true>(s[kt][nt], a0, a1, a2, a3, qf[c + e][nt][0], qf[c + e][nt][1]);
        }
      }
  }
  // scores in log2 units, hidden keys out, running maximum
  float vs[KT][2], vm = vmax;
  float mx[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = kNegInf;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    float ks[2] = {1.0f, 1.0f};
    if constexpr (FP8) {
      const float* kss = reinterpret_cast<const float*>(stage + 2 * C::kTile);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = key0 + kt * 16 + g + 8 * e;
        ks[e] = kss[r];
        vs[kt][e] = g + 8 * e < cn[kt] ? kss[kUnit + r] : 0.0f;
        vm = fmaxf(vm, vs[kt][e]);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (the two powers of two meet first: a product of a huge key's codes
        // need not fit a float before a tiny query's size is back in it)
        const float x = FP8 ? ks[j >> 1] * sq[nt][j & 1] : sq[nt][j & 1];
        s[kt][nt][j] = seen(kt, j >> 1, nt, j & 1) ? s[kt][nt][j] * x : kNegInf;
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) mx[nt][j] = fmax3(mx[nt][j], s[kt][nt][j], s[kt][nt][j + 2]);
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
  if constexpr (FP8) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
    up |= vm > vmax;
  }
  if (__any_sync(0xffffffffu, up)) {
    const float fv = FP8 && vmax > 0.0f ? vmax / vm : 1.0f;   // powers of two
    vmax = vm;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float f = m[nt][j] == kNegInf ? 0.0f : ex2(m[nt][j] - mx[nt][j]);
        m[nt][j] = mx[nt][j];
        l[nt][j] *= f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          acc[c][nt][j] *= f * fv;
          acc[c][nt][j + 2] *= f * fv;
        }
      }
  }
  // weights, their sums, and P^T as the second product's B operand
  uint32_t pf[KT][NT][2];
  float vf[KT][2];
  if constexpr (FP8) {
    // f16 weights, the largest V scale's at 2^15: a weight keeps its 11
    // bits down to 2^-29 of that scale
    const float iv = vmax > 0.0f ? 1.0f / vmax : 1.0f;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int e = 0; e < 2; ++e) vf[kt][e] = vs[kt][e] * iv * 32768.0f;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float mm[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) mm[j] = m[nt][j] == kNegInf ? 0.0f : m[nt][j];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      float p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = ex2(s[kt][nt][j] - mm[j & 1]);
        l[nt][j & 1] += p[j];
        if (FP8) p[j] *= vf[kt][j >> 1];
      }
      pf[kt][nt][0] = movm(FP8 ? pack_f16(p[0], p[1]) : pack_bf16(p[0], p[1]));
      pf[kt][nt][1] = movm(FP8 ? pack_f16(p[2], p[3]) : pack_bf16(p[2], p[3]));
    }
  }
  // O^T += V^T P^T; slots behind the last key hold anything, NaN included
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    const int c = cn[kt];
    if (c == 0) continue;
    auto product = [&](auto whole) {
      uint32_t m0 = 0xFFFFFFFFu, m1 = 0xFFFFFFFFu;
      if constexpr (!decltype(whole)::value) {
        m0 = (2 * tg < c ? 0xFFFFu : 0u) | (2 * tg + 1 < c ? 0xFFFF0000u : 0u);
        m1 = (2 * tg + 8 < c ? 0xFFFFu : 0u) | (2 * tg + 9 < c ? 0xFFFF0000u : 0u);
      }
      if constexpr (!FP8) {
#pragma unroll
        for (int cd = 0; cd < D / 16; ++cd) {
          uint32_t r[4];   // keys 0-7 by d 0-7 and 8-15, then keys 8-15
          ldsm4t(r, chunk(vbase, key0 + kt * 16 + (lane & 7) + ((lane >> 4) << 3),
                          2 * cd + ((lane >> 3) & 1)));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816<false>(acc[cd][nt], r[0] & m0, r[1] & m0, r[2] & m1, r[3] & m1,
                            pf[kt][nt][0], pf[kt][nt][1]);
        }
      } else {
#pragma unroll
        for (int cd = 0; cd < D / 16; cd += 2) {
          uint32_t r[4];   // chunk cd by keys 0-7 and 8-15, then chunk cd + 1
          ldsm4t(r, chunk(vbase, key0 + kt * 16 + (lane & 15), cd + (lane >> 4)));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // bytes (key, d), (key, d + 1), (key + 1, d), (key + 1, d + 1)
            // to the pairs of keys at d and at d + 1
            const uint32_t x = __byte_perm(r[2 * e], 0, 0x3120);
            const uint32_t y = __byte_perm(r[2 * e + 1], 0, 0x3120);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<true>(acc[cd + e][nt], e4m3_f16x2_lo(x) & m0, e4m3_f16x2_hi(x) & m0,
                             e4m3_f16x2_lo(y) & m1, e4m3_f16x2_hi(y) & m1, pf[kt][nt][0],
                             pf[kt][nt][1]);
          }
        }
      }
    };
    if (c == 16)
      product(std::true_type{});
    else
      product(std::false_type{});
  }
}

// Joins the warps, whose columns and numerators the readers below then give.  sm: maxima and sums, [warp][8 NT] each; an item's may
// still be read while the next one's are written, so items take turns.
template <class C, int D, bool FP8, int NT>
__device__ __forceinline__ void join_warps(Fold<D, NT>& f, float* join, float* sm) {
  constexpr int KW = C::kWarps;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tg = lane & 3;
  const float kNegInf = -__int_as_float(0x7f800000);
  float* sm_m = sm;
  float* sm_l = sm + C::kWarps * 8 * NT;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) f.l[nt][j] += __shfl_xor_sync(0xffffffffu, f.l[nt][j], o);
      if (g == 0) {
        sm_m[warp * 8 * NT + nt * 8 + 2 * tg + j] = f.m[nt][j];
        sm_l[warp * 8 * NT + nt * 8 + 2 * tg + j] = f.l[nt][j];
      }
    }
  compute_sync<C::kWarps>();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float mm = kNegInf;
      for (int w = 0; w < KW; ++w)
        mm = fmaxf(mm, sm_m[w * 8 * NT + nt * 8 + 2 * tg + j]);
      float x = f.m[nt][j] == kNegInf ? 0.0f : ex2(f.m[nt][j] - mm);
      if (FP8) x *= f.vmax * 3.0517578125e-5f;     // back to V's own units
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        f.acc[c][nt][j] *= x;
        f.acc[c][nt][j + 2] *= x;
      }
    }
  float* mine = join + (warp & (C::kJoin - 1)) * (C::kRegs * 32) + lane;
  for (int r = KW / C::kJoin - 1; r >= 0; --r) {
    if (warp / C::kJoin == r) {
      const bool put_first = r == KW / C::kJoin - 1;
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float* at = mine + ((c * NT + nt) * 4 + j) * 32;
            *at = put_first ? f.acc[c][nt][j] : *at + f.acc[c][nt][j];
          }
    }
    compute_sync<C::kWarps>();
  }
}
// Numerator d of column nn.
template <class C, int D, bool FP8, int NT>
__device__ __forceinline__ float joined_at(const float* join, int nn, int d) {
  const int dd = d & 15;
  const int gg = FP8 ? dd >> 1 : dd & 7, hi = FP8 ? dd & 1 : dd >> 3;
  const int at = (((d >> 4) * NT + (nn >> 3)) * 4 + hi * 2 + (nn & 1)) * 32 + gg * 4 + ((nn & 7) >> 1);
  const float* b = join + at;
  float x = b[0];
#pragma unroll
  for (int k = 1; k < C::kJoin; ++k) x += b[k * (C::kRegs * 32)];
  return x;
}
// Maximum and sum of column nn.
template <class C, int NT>
__device__ __forceinline__ void joined_state(const float* sm, int nn, float& mm, float& ll) {
  constexpr int KW = C::kWarps, N = 8 * NT;
  const float kNegInf = -__int_as_float(0x7f800000);
  const float* sm_m = sm + nn;
  const float* sm_l = sm_m + KW * N;
  mm = kNegInf;
  ll = 0.0f;
#pragma unroll
  for (int w = 0; w < KW; ++w) mm = fmaxf(mm, sm_m[w * N]);
#pragma unroll
  for (int w = 0; w < KW; ++w) {
    const float mw = sm_m[w * N];
    ll += mw == kNegInf ? 0.0f : ex2(mw - mm) * sm_l[w * N];
  }
}

template <int D, bool FP8, int NT, bool SPARSE>
__global__ void __launch_bounds__(Cfg<D, FP8, NT>::kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                      const CacheArgs a) {
  using C = Cfg<D, FP8, NT>;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
  constexpr int NH = 8 * NT;                       // query heads of an item
  constexpr int KT = C::kKT, kUnit = C::kUnit, kGroups = kUnit / 16;
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

  if (SPARSE && a.row_flags && !a.row_flags[a.T]) return;   // no row to do again
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
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
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
    if (lane == 31) misc[8 + warp] = inc;
    __syncthreads();
    int base = inc - sum;
    for (int w = 0; w < warp; ++w) base += misc[8 + w];
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
  Cursor<SPARSE, kUnit> cur;
  cur.start(a, pre, rows, HX, u0);

  // with row flags, items of rows without one are passed over
  auto skip = [&](int& i) -> bool {
    if (!SPARSE || !a.row_flags || a.row_flags[cur.row]) return false;
    i += cur.units - 1 - cur.k;
    cur.k = cur.units - 1;
    if (i + 1 < n_units) cur.next(a, pre, HX);
    return true;
  };

  if (warp == kWarps) {
    // ---- loads: lane i brings page i of the unit ----
    const int ppu = kUnit >> a.ps_log2;
    int row = -1, s = 0, len = 0;
    int issued = 0;
    for (int i = 0; i < n_units; ++i) {
      if (skip(i)) continue;
      const int st = issued % C::kStages;
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
      if (issued >= C::kStages && !mbar_wait(&empty[st], ((issued / C::kStages) - 1) & 1, abort, 1)) break;
      unsigned char* stage = smem + st * C::kStageStep;
      const int v16 = __shfl_sync(0xffffffffu, vc, (lane & (kGroups - 1)) >> (a.ps_log2 - 4));
      if (lane < kGroups)
        cnt[st * kGroups + lane] = min(16, max(0, v16 - 16 * (lane & ((1 << (a.ps_log2 - 4)) - 1))));
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
      ++issued;
      if (i + 1 < n_units) cur.next(a, pre, HX);
    }
    // nothing may still be writing shared memory when the CTA ends, whoever's
    // wait ran out (the flag may rise after this warp has looked)
    for (int i = max(0, issued - C::kStages); i < issued; ++i)
      mbar_wait_drain(&full[i % C::kStages], (i / C::kStages) & 1);
    return;
  }

  // ---- compute ----
  const int g = lane >> 2;
  const float sc = a.scale_log2;
  Fold<D, NT> f;
  float* join = reinterpret_cast<float*>(smem + C::oJoin);
  const float kNegInf = -__int_as_float(0x7f800000);
  bool fresh = true;                               // no unit of the item taken yet
  int k_first = 0;                                 // first unit of the item in this run
  int turn = 0;
  float* sm_m = sm_m0;

  int taken = 0;
  for (int i = 0; i < n_units; ++i) {
    if (skip(i)) continue;
    const int st = taken % C::kStages;
    const int hk = cur.hx / HG, h0 = hk * a.G + (cur.hx - hk * HG) * NH;
    const int nh = min(NH, (hk + 1) * a.G - h0);   // heads in use
    if (fresh) {
      fresh = false;
      k_first = cur.k;
      f.vmax = 0.0f;
      const __nv_bfloat16* q = a.q + (int64_t)cur.row * a.sq_t + (int64_t)h0 * a.sq_h;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        fold_query<D, FP8, NT>(f, nt, q + (int64_t)(nt * 8 + g) * a.sq_h, nt * 8 + g < nh, sc);
    }
    const bool ok = mbar_wait(&full[st], (taken / C::kStages) & 1, abort, 2);
    ++taken;
    int cn[KT], any = 0;                           // keys of this warp's tiles
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      cn[kt] = ok ? cnt[st * kGroups + KT * warp + kt] : 0;
      any |= cn[kt];
    }
    if (any) {
      fold_unit<C, D, FP8, NT>(f, smem + st * C::kStageStep, warp * 16 * KT, cn,
                               [&](int kt, int e, int, int) { return g + 8 * e < cn[kt]; });
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);

    if (cur.k + 1 == cur.units || i + 1 == n_units) {
      // ---- join the computing warps ----
      join_warps<C, D, FP8, NT>(f, join, sm_m);
      auto joined = [&](int nn, int d) { return joined_at<C, D, FP8, NT>(join, nn, d); };
      auto state = [&](int nn, float& mm, float& ll) { joined_state<C, NT>(sm_m, nn, mm, ll); };
      __nv_bfloat16* out = a.o + (int64_t)cur.row * a.so_t + (int64_t)h0 * a.so_h;
      auto put = [&](int nn, int d, float x, float y, float mm, float ll) {
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        *reinterpret_cast<uint32_t*>(out + (int64_t)nn * a.so_h + d) = pack_bf16(x * inv, y * inv);
        if (d == 0 && a.lse)
          a.lse[(int64_t)cur.row * a.H + h0 + nn] =
              ll == 0.0f ? kNegInf : (mm + log2f(ll)) * 0.6931471805599453f;
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
        compute_sync<C::kWarps>();
        if (tid == 0)
          misc[1] = atomicInc(reinterpret_cast<unsigned int*>(a.counters) + cf, (unsigned)(cl - cf)) ==
                    (unsigned)(cl - cf);
        compute_sync<C::kWarps>();
        if (misc[1]) {
          __threadfence();
          for (int e = tid; e < nh * (D / 2); e += 32 * kWarps) {
            const int nn = e / (D / 2), d = 2 * (e - nn * (D / 2));
            float mm = kNegInf, ll = 0.0f, x = 0.0f, y = 0.0f;
            for (int c0 = cf; c0 <= cl; c0 += 8) {         // 8 parts' loads in flight
              float pm[8], pl[8];
              float2 pv[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int c = min(c0 + k, cl), sl = 2 * c + (c == cf);
                pm[k] = __ldcg(a.part_ml + sl * (2 * kMaxTileHeads) + nn);
                pl[k] = __ldcg(a.part_ml + sl * (2 * kMaxTileHeads) + kMaxTileHeads + nn);
                pv[k] = __ldcg(reinterpret_cast<const float2*>(a.part_o + (int64_t)sl * (kMaxTileHeads * 128) + nn * D + d));
              }
              float top = mm;
#pragma unroll
              for (int k = 0; k < 8; ++k) top = fmaxf(top, pm[k]);
              const float old = mm == kNegInf ? 0.0f : ex2(mm - top);
              mm = top;
              ll *= old;
              x *= old;
              y *= old;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float f = pm[k] == kNegInf || c0 + k > cl ? 0.0f : ex2(pm[k] - mm);
                ll += f * pl[k];
                x += f * pv[k].x;
                y += f * pv[k].y;
              }
            }
            put(nn, d, x, y, mm, ll);
          }
        }
      }
      fresh = true;
      turn ^= 1;
      sm_m = sm_m0 + turn * (2 * C::kWarps * 8 * NT);
    }
    if (i + 1 < n_units) cur.next(a, pre, HX);
  }
}

// ---------------------------------------------------------------------------
// Sparse attention of many rows
// ---------------------------------------------------------------------------
// Rows next to each other read mostly the same pages, and one at a time they
// are bound by what the L2 cache delivers (1332 rows of 1024 keys: 595 us).  So
// up to 128 (row, query head) pairs of a sequence share their loads: a first
// kernel joins their lists, each page with the bits of the rows that read it,
// and the pairs of the other rows see none of its keys.
//
// A weight of zero times a value that is not finite would spoil the columns
// that do not see it.  Rows with a result that is not finite are therefore
// flagged and done again on their own, where hidden keys are never multiplied.

// Joint page lists, pages in order.  Where a row lists a page twice, the
// tile's lists stand one after the other instead, so that it counts twice.
__global__ void __launch_bounds__(256) cache_lists_kernel(const CacheArgs a) {
  extern __shared__ uint32_t bits[];   // rows that read a page, for each page
  __shared__ int wsum[8];
  __shared__ int twice;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hk = blockIdx.y;
  const RowTile tile = row_tile(a, blockIdx.x, a.tile_rows);
  const int64_t item = (int64_t)blockIdx.x * a.Hkv + hk;
  if (hk == 0 && blockIdx.x == 0) {
    for (int i = tid; i < kMaxTileParts; i += 256) a.tile_arrived[i] = 0;
    if (tid == 0) a.row_flags[a.T] = 0;
  }
  if (hk == 0)
    for (int t = tile.t0 + tid; t < tile.t1; t += 256) {
      a.row_flags[t] = 0;
      row_pos(a, t, tile.s);           // (reports a row without a position)
    }
  if (tile.t0 >= tile.t1) return;
  const int len = seq_len(a, tile.s);
  const int pages = (len + a.page_size - 1) >> a.ps_log2, rows = tile.t1 - tile.t0;
  for (int j = tid; j < pages; j += 256) bits[j] = 0;
  if (tid == 0) twice = 0;
  __syncthreads();
  // row r sees the pages up to its own
  const int64_t pos0 = (int64_t)len - (a.cu[tile.s + 1] - tile.t0);
  auto entry = [&](int i, int& r) -> int {
    r = i / a.n_select;
    const int e = a.sel[((int64_t)(tile.t0 + r) * a.Hkv + hk) * a.n_select + (i - r * a.n_select)];
    return e >= 0 && e < pages && (int64_t)e << a.ps_log2 <= pos0 + r ? e : -1;
  };
  for (int i = tid; i < rows * a.n_select; i += 256) {
    int r;
    const int e = entry(i, r);
    if (e >= 0 && atomicOr(&bits[e], 1u << r) >> r & 1) twice = 1;
  }
  __syncthreads();
  int2* out = a.lists + item * a.list_cap;
  if (twice) {
    for (int i = tid; i < rows * a.n_select; i += 256) {
      int r;
      const int e = entry(i, r);
      out[i] = make_int2(max(e, 0), e >= 0 ? 1 << r : 0);
    }
    if (tid == 0) a.list_n[item] = rows * a.n_select;
    return;
  }
  int at = 0;
  for (int base = 0; base < pages; base += 256) {
    const int j = base + tid;
    const uint32_t m = j < pages ? bits[j] : 0u;
    const uint32_t b = __ballot_sync(0xffffffffu, m != 0);
    __syncthreads();
    if (lane == 0) wsum[warp] = __popc(b);
    __syncthreads();
    int k = at;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) k += wsum[w];
      at += wsum[w];
    }
    if (m) out[k + __popc(b & ((1u << lane) - 1))] = make_int2(j, (int)m);
  }
  if (tid == 0) a.list_n[item] = at;
}

// Tiles of up to 128 (row, query head) pairs on tcgen05: the pairs are the 128
// rows of S = Q K^T and O += P V, two threads of the softmax share one of them
// (64 keys each), S and P (bf16, over S's own columns) and O stand in TMEM.  A
// block has one K and one V buffer: K of the next unit loads while this one's
// softmax runs, V while the next S does, and two blocks share an SM.
//
// Codes of FP8 caches load into the upper half of their buffer, and the softmax
// threads widen them in place to bf16 with the scale multiplied in, which is
// exact (4 significant bits, scales are powers of two).  Their weights are bf16
// here, as V is; few rows' are f16 (cache_attn_kernel), which holds 3 bits more.
//
// The tiles that are left after whole rounds of the GPU's places are cut along
// their keys, so that the last round is full too: their parts meet in the
// workspace, and the block that arrives last joins them in order.
//
// 1332 rows of 32 query heads, 1024 keys each, bf16: 115 us with the lists,
// FP8 143; 131 without the cut, 145 with one thread a pair.  A tile's
// blocks wait for one another's steps (S, softmax, O) and two blocks an SM
// cover a part of it: the tensor pipe is busy a quarter of the time.  Units of 64
// keys with a second S, multiplied ahead of the softmax, took 13 us more.
//
// A row's greatest weight is exactly 1, so P's rounding spares it (letting the
// maximum lag and O be rescaled seldom was 7 percent faster and a fifth less
// exact where few keys carry a row).
template <int D>
struct TileSmem {
  static constexpr int kRows = 128 * 128;          // bytes of 128 rows by 64 elements
  static constexpr int kOp = D / 64 * kRows;       // one operand
  static constexpr int oQ = 0, oK = kOp, oV = 2 * kOp;
  static constexpr int oInfo = 3 * kOp;            // [2][8] int4: the pages of a unit
  static constexpr int oMax = oInfo + 256;         // [2][2][128] maxima of a row's halves, then sums
  static constexpr int oScale = oMax + 2048;       // FP8: [2][128] scales of K and V
  static constexpr int oBar = oScale + 1024;
  static constexpr int kBytes = oBar + 64 + 1024;  // 1024 to align
};

// This thread's half row of codes to bf16 times `scale` (zeros where !keep), in
// place: the codes stand in the tile's upper half, all 256 threads read them
// before any writes.
template <int D>
__device__ __forceinline__ void widen(unsigned char* tile, int key, int half, float scale, bool keep) {
  using L = TileSmem<D>;
  constexpr int N = D / 32;                        // chunks of 16 codes
  uint4 w[N];
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const int x = half * N + c;
    w[c] = *reinterpret_cast<const uint4*>(tile + L::kOp / 2 + key * D +
                                           ((x ^ (D == 128 ? key & 7 : (key >> 1) & 3)) << 4));
  }
  asm volatile("bar.sync 5, 256;" ::: "memory");
  auto two = [&](uint32_t f16x2) -> uint32_t {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f16x2));
    return keep ? pack_bf16(v.x * scale, v.y * scale) : 0u;
  };
#pragma unroll
  for (int c = 0; c < N; ++c)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int y = 2 * (half * N + c) + e;
      const uint32_t u = e ? w[c].z : w[c].x, v = e ? w[c].w : w[c].y;
      *reinterpret_cast<uint4*>(tile + (y >> 3) * L::kRows + key * 128 + (((y & 7) ^ (key & 7)) << 4)) =
          make_uint4(two(e4m3_f16x2_lo(u)), two(e4m3_f16x2_hi(u)), two(e4m3_f16x2_lo(v)), two(e4m3_f16x2_hi(v)));
    }
  fence_proxy_async_smem();
}

template <int D, bool FP8>
__global__ void __launch_bounds__(320, 2)
    cache_tile_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                      const CacheArgs a, int whole_items, int cuts) {
  using L = TileSmem<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int over = max(0, (int)blockIdx.x - whole_items);
  const int64_t item = (int)blockIdx.x < whole_items ? (int)blockIdx.x : whole_items + over / cuts;
  const int hk = (int)(item % a.Hkv);
  const RowTile tile = row_tile(a, (int)(item / a.Hkv), a.tile_rows);
  if (tile.t0 >= tile.t1) return;
  const int n = a.list_n[item], ppu = 128 >> a.ps_log2, all_units = max(1, (n + ppu - 1) / ppu);
  // this block's units: all of them, or part `cut` of `parts`
  const int parts = (int)blockIdx.x < whole_items ? 1 : min(cuts, all_units);
  const int cut = (int)blockIdx.x < whole_items ? 0 : over % cuts;
  if (cut >= parts) return;
  const int unit0 = (int)((int64_t)all_units * cut / parts);
  const int units = (int)((int64_t)all_units * (cut + 1) / parts) - unit0;
  const int len = seq_len(a, tile.s), t0 = tile.t0, pairs = (tile.t1 - t0) * a.G;

  int4* info = reinterpret_cast<int4*>(smem + L::oInfo);   // first position, rows' bits, keys that exist
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::oBar);
  uint64_t *full_k = bars, *full_v = bars + 1, *s_ready = bars + 2, *p_ready = bars + 3, *o_done = bars + 4,
           *k_ready = FP8 ? bars + 5 : full_k,             // K in bf16
           *seen = bars + 5;                               // bf16: the softmax warps know that K is there
  uint32_t* slot = reinterpret_cast<uint32_t*>(bars + 6);
  int* flag = reinterpret_cast<int*>(bars + 7);            // [0]: a wait gave up, [1]: the last part
  float* scales = reinterpret_cast<float*>(smem + L::oScale);
  const AbortCtx abort{flag, a.status};
  if (tid == 0) {
    mbar_init(full_k, 1);
    mbar_init(full_v, 1);
    mbar_init(s_ready, 1);
    mbar_init(p_ready, 256);
    mbar_init(o_done, 1);
    mbar_init(bars + 5, FP8 ? 256 : 8);
    *flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(slot, 256);
    tmem_relinquish();
  }
  // pair i of the tile: row i / G, query head i % G of the key head
  const int pair = tid & 127, half = tid >> 7;             // (softmax threads)
  const int r = pair / a.G, h = hk * a.G + pair - r * a.G;
  if (tid < 256) {
    const __nv_bfloat16* q = a.q + (int64_t)(t0 + r) * a.sq_t + (int64_t)h * a.sq_h;
    constexpr int N = D / 16;                              // chunks of half a row
    uint4 w[N];
#pragma unroll
    for (int c = 0; c < N; ++c)
      w[c] = pair < pairs ? *reinterpret_cast<const uint4*>(q + 8 * (half * N + c)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const int x = half * N + c;
      *reinterpret_cast<uint4*>(smem + L::oQ + (x >> 3) * L::kRows + pair * 128 + (((x & 7) ^ (pair & 7)) << 4)) = w[c];
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tS = *slot, tO = tS + 128;

  if (warp == 8) {
    // ---- loads: lane i brings page i of the unit ----
    const int2* list = a.lists + item * a.list_cap;
    bool ok = true;
    int nk = 0, nv = 0;                // phases that full_k and full_v were given
    for (int i = 0; i < units; ++i) {
      const int at = (unit0 + i) * ppu + lane;
      const int2 e = lane < ppu && at < n ? list[at] : make_int2(0, 0);
      int vc = e.y ? min(a.page_size, max(0, len - (e.x << a.ps_log2))) : 0, page = 0;
      if (vc > 0) {
        page = page_of(a, tile.s, e.x);
        if (page < 0) vc = 0;
      }
      const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, vc > 0)) * a.page_size * (FP8 ? D + 4 : 2 * D);
      // K is free; and (FP8: as S tells) no softmax warp still waits for full_k's
      // last phase, which a next one, done early, would hide from it
      if (i > 0) ok = mbar_wait(s_ready, (i - 1) & 1, abort, 1) && (FP8 || mbar_wait(seen, (i - 1) & 1, abort, 10));
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane < ppu) info[(i & 1) * 8 + lane] = make_int4(e.x << a.ps_log2, e.y, vc, 0);
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(full_k, bytes);
      ++nk;
      __syncwarp();
      const int off = lane << a.ps_log2;
      if (vc > 0) {
        if constexpr (FP8) {
          tma_load_4d(smem + L::oK + L::kOp / 2 + off * D, &mk, full_k, 0, 0, hk, page);
          bulk_load(scales + off, a.k_scale + (((int64_t)page * a.Hkv + hk) << a.ps_log2), a.page_size * 4, full_k);
        } else {
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(smem + L::oK + c * L::kRows + off * 128, &mk, full_k, c * 64, 0, hk, page);
        }
      }
      if (i > 0) ok = mbar_wait(o_done, (i - 1) & 1, abort, 2);        // V is free
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) mbar_arrive_expect_tx(full_v, bytes);
      ++nv;
      __syncwarp();
      if (vc > 0) {
        if constexpr (FP8) {
          tma_load_4d(smem + L::oV + L::kOp / 2 + off * D, &mv, full_v, 0, 0, hk, page);
          bulk_load(scales + 128 + off, a.v_scale + (((int64_t)page * a.Hkv + hk) << a.ps_log2), a.page_size * 4, full_v);
        } else {
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(smem + L::oV + c * L::kRows + off * 128, &mv, full_v, c * 64, 0, hk, page);
        }
      }
    }
    // nothing may still be writing shared memory when the block ends, whatever
    // wait of whichever role ran out
    if (nk) mbar_wait_drain(full_k, (nk - 1) & 1);
    if (nv) mbar_wait_drain(full_v, (nv - 1) & 1);
  } else if (warp == 9) {
    // ---- products ----
    if (lane == 0) {
      const uint32_t sq = smem_u32(smem + L::oQ), sk = smem_u32(smem + L::oK), sv = smem_u32(smem + L::oV);
      constexpr uint32_t idesc_s = idesc_bf16(128, 128, false), idesc_o = idesc_bf16(128, D, true);
      int ns = 0, no = 0;              // products committed to s_ready and o_done
      for (int i = 0; i < units; ++i) {
        // (S's columns are free: they held P of the unit before, whose product
        // is ahead in the pipe)
        if (!mbar_wait(k_ready, i & 1, abort, 3)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_f16_ss(tS, smem_desc_sw128(sq + (kk >> 2) * L::kRows + (kk & 3) * 32, 16, 1024),
                     smem_desc_sw128(sk + (kk >> 2) * L::kRows + (kk & 3) * 32, 16, 1024), idesc_s, kk > 0 ? 1u : 0u);
        tc_commit(s_ready);
        ++ns;
        if (!mbar_wait(p_ready, i & 1, abort, 4) || !mbar_wait(full_v, i & 1, abort, 5)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_f16_ts(tO, tS + kk * 8, smem_desc_sw128(sv + kk * 16 * 128, L::kRows, 1024), idesc_o,
                     (i > 0 || kk > 0) ? 1u : 0u);
        tc_commit(o_done);
        ++no;
      }
      // nor may a product read that memory, or write the columns given back
      if (ns) mbar_wait_drain(s_ready, (ns - 1) & 1);
      if (no) mbar_wait_drain(o_done, (no - 1) & 1);
    }
  } else {
    // ---- softmax: two threads have a pair, 64 keys of a unit each ----
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tH = tS + lanes + half * 64;            // this half's scores
    const float sc = a.scale_log2, big = __int_as_float(0x7f800000);
    const uint32_t bit = pair < pairs ? 1u << r : 0u;
    const int pos0 = len - (a.cu[tile.s + 1] - t0);
    const int sees = min(pos0 + r, len - 1) + 1;           // keys that the row sees
    float* maxima = reinterpret_cast<float*>(smem + L::oMax);
    // the two warps of 32 pairs meet (64 threads; every one of them passes here
    // the same number of times, whatever a wait says)
    auto meet = [&] { asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory"); };
    float m = -big, l = 0.0f;
    bool ok = true;
    for (int i = 0; i < units; ++i) {
      ok = ok && mbar_wait(full_k, i & 1, abort, 6);
      if constexpr (FP8) {
        widen<D>(smem + L::oK, pair, half, scales[pair], true);
        if (ok) mbar_arrive(k_ready);                      // (else no product may start on it)
      } else {
        __syncwarp();                                      // (every lane has waited)
        if (lane == 0) mbar_arrive(seen);
      }
      ok = ok && mbar_wait(s_ready, i & 1, abort, 7);
      tc_fence_after();
      const int4* pages = info + (i & 1) * 8;
      // visible keys of each 32
      uint32_t vis[2];
      bool whole = true;                                   // every slot of the half holds a key
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        vis[c] = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {                      // 16 keys at a time: one page
          const int k = half * 64 + c * 32 + e * 16;
          const int4 w = pages[k >> a.ps_log2];
          const int first = k & (a.page_size - 1);
          const int seen = (w.y & bit) ? min(w.z, sees - w.x) - first : 0;
          vis[c] |= (seen >= 16 ? 0xFFFFu : seen > 0 ? (1u << seen) - 1 : 0u) << (16 * e);
          whole &= w.z == a.page_size;
        }
      }
      const bool live = __all_sync(0xffffffffu, ok);
      const bool any = __any_sync(0xffffffffu, vis[0] | vis[1]) && live;
      float mx = -big;
      auto top = [&](const uint32_t (&x)[32], uint32_t v) {
        if (v == 0xFFFFFFFFu) {
#pragma unroll
          for (int k = 0; k < 32; k += 2) mx = fmax3(mx, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
        } else if (v) {
#pragma unroll
          for (int k = 0; k < 32; ++k) mx = fmaxf(mx, v >> k & 1 ? __uint_as_float(x[k]) : -big);
        }
      };
      if (any) {
        uint32_t x[32], y[32];
        tmem_ld32x2(tH, tH + 32, x, y);
        top(x, vis[0]);
        top(y, vis[1]);
      }
      float* mine = maxima + (i & 1) * 256;
      mine[half * 128 + pair] = mx;
      meet();
      mx = fmaxf(mx, mine[(half ^ 1) * 128 + pair]) * sc;
      const bool move = mx > m;
      if (__any_sync(0xffffffffu, move)) {
        const float f = !move ? 1.0f : m == -big ? 0.0f : ex2(m - mx);
        if (move) m = mx;
        l *= f;
        if (i > 0 && live) {           // (the last product is done: S came after it)
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint32_t at = tO + lanes + half * (D / 2) + c * 32;
            uint32_t o[32];
            tmem_ld32(at, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st32(at, o);
          }
        }
      }
      const float mm = m == -big ? 0.0f : m;
      // P of both halves lies over S's first 64 columns: every score is read
      // (into P's registers) before any P is written
      uint32_t p[2][16];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int k = 0; k < 16; ++k) p[c][k] = 0u;
        if (!any || !__any_sync(0xffffffffu, vis[c])) continue;
        uint32_t x[32];
        tmem_ld32(tH + c * 32, x);
        // (uniform) some row sees a part of the 32 keys, or there are slots
        // without one; else a row sees all of them or none
        const bool part = !whole || __any_sync(0xffffffffu, vis[c] + 1u > 1u);
        const float off = vis[c] ? mm : big;               // (none: 2^-inf)
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          float u = ex2(fmaf(__uint_as_float(x[k]), sc, -off)), v = ex2(fmaf(__uint_as_float(x[k + 1]), sc, -off));
          if (part) {
            u = vis[c] >> k & 1 ? u : 0.0f;
            v = vis[c] >> (k + 1) & 1 ? v : 0.0f;
          }
          l += u + v;
          p[c][k / 2] = pack_bf16(u, v);
        }
      }
      tc_fence_before();
      meet();
      tc_fence_after();
      tmem_st16(tS + lanes + half * 32, p[0]);
      tmem_st16(tS + lanes + half * 32 + 16, p[1]);
      tmem_wait_st();
      if constexpr (FP8) {
        ok = ok && mbar_wait(full_v, i & 1, abort, 8);
        const int4 w = pages[pair >> a.ps_log2];
        widen<D>(smem + L::oV, pair, half, scales[128 + pair], (pair & (a.page_size - 1)) < w.z);
      } else if (!whole) {
        // slots without a key hold anything: as zeros, P's zeros leave O alone
        ok = ok && mbar_wait(full_v, i & 1, abort, 8);
        const int key = half * 64 + (tid & 63);            // (two threads a key: half a row each)
        const int4 w = pages[key >> a.ps_log2];
        if (ok && (key & (a.page_size - 1)) >= w.z)
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const int x = (pair >> 6) * (D / 16) + c;
            *reinterpret_cast<uint4*>(smem + L::oV + (x >> 3) * L::kRows + key * 128 + (x & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      mbar_arrive(p_ready);
    }
    ok = ok && mbar_wait(o_done, (units - 1) & 1, abort, 9);
    float* sums = maxima + (units & 1) * 256;
    sums[half * 128 + pair] = l;
    meet();
    l += sums[(half ^ 1) * 128 + pair];
    float o[D / 2];                                        // the thread's half of O's row
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t x[32];
        tmem_ld32(tO + lanes + half * (D / 2) + c * 32, x);
#pragma unroll
        for (int k = 0; k < 32; ++k) o[c * 32 + k] = __uint_as_float(x[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < D / 2; ++k) o[k] = 0.0f;
    }
    bool put = true;
    if (parts > 1) {
      // (thread-major: neighbouring threads' numbers stand next to each other)
      float* mine = a.tile_parts + (int64_t)over * (256 * (D / 2 + 2)) + tid;
#pragma unroll
      for (int k = 0; k < D / 2; ++k) __stcg(mine + k * 256, o[k]);
      __stcg(mine + (D / 2) * 256, m);
      __stcg(mine + (D / 2 + 1) * 256, l);
      __threadfence();
      asm volatile("bar.sync 5, 256;" ::: "memory");
      if (tid == 0)
        flag[1] = atomicInc(reinterpret_cast<unsigned int*>(a.tile_arrived) + over / cuts, (unsigned)(parts - 1)) ==
                  (unsigned)(parts - 1);
      asm volatile("bar.sync 5, 256;" ::: "memory");
      put = flag[1];
      if (put) {
        __threadfence();
        const float* first = a.tile_parts + (int64_t)(over - cut) * (256 * (D / 2 + 2)) + tid;
        m = -big;
        l = 0.0f;
        for (int q = 0; q < parts; ++q)
          m = fmaxf(m, __ldcg(first + (int64_t)q * (256 * (D / 2 + 2)) + (D / 2) * 256));
#pragma unroll
        for (int k = 0; k < D / 2; ++k) o[k] = 0.0f;
        for (int q = 0; q < parts; ++q) {
          const float* part = first + (int64_t)q * (256 * (D / 2 + 2));
          const float mq = __ldcg(part + (D / 2) * 256), f = mq == -big ? 0.0f : ex2(mq - m);
          l += f * __ldcg(part + (D / 2 + 1) * 256);
#pragma unroll
          for (int k = 0; k < D / 2; ++k) o[k] += f * __ldcg(part + k * 256);
        }
      }
    }
    if (put && pair < pairs) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      bool fine = l < big && m < big;
      __nv_bfloat16* out = a.o + (int64_t)(t0 + r) * a.so_t + (int64_t)h * a.so_h + half * (D / 2);
#pragma unroll
      for (int k = 0; k < D / 2; k += 8) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] = o[k + e] * inv;
          fine &= fabsf(y[e]) < big;
        }
        *reinterpret_cast<uint4*>(out + k) =
            make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
      }
      if (!fine) a.row_flags[t0 + r] = a.row_flags[a.T] = 1;
      if (half == 0 && a.lse)
        a.lse[(int64_t)(t0 + r) * a.H + h] = l == 0.0f ? -big : (m + log2f(l)) * 0.6931471805599453f;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tS, 256);
}

template <int D, bool FP8, int NT, bool SPARSE>
cudaError_t run(const CacheArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  using C = Cfg<D, FP8, NT>;
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(dev, sms);
  if (e != cudaSuccess) return e;
  const int bytes = C::kBytes + (SPARSE ? 0 : (a.S + 1) * 4);
  static_assert(C::kBytes + (SPARSE ? 0 : (kMaxDecodeSeqs + 1) * 4) <= 232448, "shared memory");
  auto k = cache_attn_kernel<D, FP8, NT, SPARSE>;
  static OncePerDevice once;
  e = once.allow(reinterpret_cast<const void*>(k), dev, C::kBytes + (SPARSE ? 0 : (kMaxDecodeSeqs + 1) * 4));
  if (e != cudaSuccess) return e;
  constexpr int kUnit = C::kUnit;
  // no more CTAs than units the call can have
  const int64_t HX = (int64_t)a.Hkv * ((a.G + 8 * NT - 1) / (8 * NT));
  const int64_t per = ((int64_t)(SPARSE ? a.n_select : a.max_pages) * a.page_size + kUnit - 1) / kUnit;
  int64_t grid = (SPARSE ? a.T : a.S) * HX * per;
  if (grid > sms) grid = sms;
  if (grid > kMaxAttnCtas) grid = kMaxAttnCtas;
  k<<<(int)grid, C::kThreads, bytes, s>>>(mk, mv, a);
  return cudaGetLastError();
}

template <int D, bool FP8>
cudaError_t pick(const CacheArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, bool sparse,
                 cudaStream_t s) {
  // Groups of more than 8 query heads take two column tiles where the cache's
  // bytes bound, so that each key is read once for up to 16 of them; with fewer
  // units than that a second tile only lengthens an item's chain.  16 heads a
  // key head: 12 units 13.7 us with two tiles and 9.5 with one, 1000 units 34
  // and 26, 4000 units 50 and 53, 16000 units 123 and 211; FP8 2000 units 49
  // and 42, 4000 units 66 and 62, 8000 units 118 and 125.
  int dev = 0, sms = 0;
  const cudaError_t e = device_sms(dev, sms);
  if (e != cudaSuccess) return e;
  constexpr int kUnit = Cfg<D, FP8, 1>::kUnit;
  static_assert(kUnit == Cfg<D, FP8, 2>::kUnit, "units are counted alike");
  const int64_t pages = !sparse ? a.max_pages : a.n_select < a.max_pages ? a.n_select : a.max_pages;
  const int64_t units = (sparse ? a.T : a.S) * (int64_t)a.Hkv * ((pages * a.page_size + kUnit - 1) / kUnit);
  if (a.G <= 8 || units <= (FP8 ? 32 : 16) * sms)
    return sparse ? run<D, FP8, 1, true>(a, mk, mv, s) : run<D, FP8, 1, false>(a, mk, mv, s);
  return sparse ? run<D, FP8, 2, true>(a, mk, mv, s) : run<D, FP8, 2, false>(a, mk, mv, s);
}

}  // namespace

static cudaError_t run_lists(const CacheArgs& a, int64_t tiles, int dev, cudaStream_t s) {
  static OncePerDevice once;
  const cudaError_t e = once.allow(reinterpret_cast<const void*>(cache_lists_kernel), dev, kMaxSelectPages * 4);
  if (e != cudaSuccess) return e;
  cache_lists_kernel<<<dim3((unsigned)tiles, a.Hkv), 256, a.max_pages * 4, s>>>(a);
  return cudaGetLastError();
}

template <int D, bool FP8>
static cudaError_t run_tiles(const CacheArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int64_t tiles,
                             int sms, int dev, cudaStream_t s) {
  static OncePerDevice once;
  auto k = cache_tile_kernel<D, FP8>;
  const cudaError_t e = once.allow(reinterpret_cast<const void*>(k), dev, TileSmem<D>::kBytes);
  if (e != cudaSuccess) return e;
  // whole rounds of two blocks an SM; the items left are cut so that they fill
  // one more (into 8 parts at most, of which a part has a few units)
  const int64_t items = tiles * a.Hkv, places = 2 * sms < kMaxTileParts ? 2 * sms : kMaxTileParts;
  const int64_t whole = items / places * places, left = items - whole;
  int cuts = left ? (int)(places / left) : 1;
  if (cuts > 8) cuts = 8;
  k<<<(unsigned)(cuts > 1 ? whole + left * cuts : items), 320, TileSmem<D>::kBytes, s>>>(
      mk, mv, a, (int)(cuts > 1 ? whole : items), cuts);
  return cudaGetLastError();
}

cudaError_t launch_cache_attn(const CacheArgs& args, const CUtensorMap& mk, const CUtensorMap& mv,
                              bool sparse, cudaStream_t s) {
  CacheArgs a = args;
  a.row_flags = nullptr;
  // Rows together where there are enough for what the lists and the parts cost:
  // bf16, 8 key heads of 4 query heads, 16 pages of 64 keys: 43 rows took 31 us
  // either way, 75 rows 45 us on their own and 37 together, 183 rows 92 and 40.
  // FP8's codes are widened, which 75 rows (40 and 42 us) do not earn back and
  // 183 (81 and 45) do.
  if (sparse && a.cu) {
    int dev = 0, sms = 0;
    cudaError_t e = device_sms(dev, sms);
    if (e != cudaSuccess) return e;
    const int rows = tile_rows(a.G, a.T, a.S, a.max_pages);
    const int64_t tiles = rows ? tile_count(rows, a.T, a.S) : 0;
    if (rows && (int64_t)a.T * a.Hkv >= (a.fp8 ? 4 : 2) * sms && tiles * a.Hkv < 0x7fffffff) {
      a.tile_rows = rows;
      a.list_cap = rows * a.n_select;
      a.tile_parts = reinterpret_cast<float*>(a.scratch);
      a.lists = reinterpret_cast<int2*>(reinterpret_cast<char*>(a.scratch) + tile_part_bytes(tiles * a.Hkv));
      a.list_n = reinterpret_cast<int*>(a.lists + tiles * a.Hkv * a.list_cap);
      a.tile_arrived = a.list_n + tiles * a.Hkv;
      a.row_flags = a.tile_arrived + kMaxTileParts;
      e = run_lists(a, tiles, dev, s);
      if (e == cudaSuccess) {
        if (a.d == 128)
          e = a.fp8 ? run_tiles<128, true>(a, mk, mv, tiles, sms, dev, s) : run_tiles<128, false>(a, mk, mv, tiles, sms, dev, s);
        else
          e = a.fp8 ? run_tiles<64, true>(a, mk, mv, tiles, sms, dev, s) : run_tiles<64, false>(a, mk, mv, tiles, sms, dev, s);
      }
      if (e != cudaSuccess) return e;
    }
  }
  if (a.d == 128)
    return a.fp8 ? pick<128, true>(a, mk, mv, sparse, s) : pick<128, false>(a, mk, mv, sparse, s);
  return a.fp8 ? pick<64, true>(a, mk, mv, sparse, s) : pick<64, false>(a, mk, mv, sparse, s);
}

}  // namespace ta
