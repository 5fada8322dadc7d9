// ta_cache_api.cu -- the C ABI of the cached-attention operators: argument
// validation, the workspace, TMA descriptors of the cache and the launches.
#include <cmath>

#include "ta_cache.cuh"

namespace {

using ta::CacheArgs;

bool aligned(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }

ta_status validate(const ta_cache_params* p) {
  if (!p) return TA_ERR_INVALID_ARG;
  if (p->n_pages < 1 || p->H < 1 || p->Hkv < 1 || p->H % p->Hkv || p->S < 1 || p->T < 1 ||
      p->max_pages < 1)
    return TA_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return TA_ERR_UNSUPPORTED;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128)
    return TA_ERR_UNSUPPORTED;
  if (p->format != TA_CACHE_BF16 && p->format != TA_CACHE_FP8) return TA_ERR_INVALID_ARG;
  if (p->n_select < 0 || p->n_first < 0 || p->rot_dim < 0 || p->rot_dim > p->d || p->rot_dim % 16 ||
      p->rot_rows < 0 || (p->rot_interleaved != 0 && p->rot_interleaved != 1))
    return TA_ERR_INVALID_ARG;
  if (p->n_select > 0 &&
      (p->n_recent < 1 || (int64_t)p->n_first + p->n_recent > p->n_select))
    return TA_ERR_INVALID_ARG;
  if (!std::isfinite(p->softmax_scale) || p->softmax_scale < 0.0f) return TA_ERR_INVALID_ARG;
  // positions, grid dimensions and the decode kernel's unit counts fit 31 bits
  if ((int64_t)p->max_pages * p->page_size > (1 << 30) || p->H > 32768 || p->n_select > 1024 ||
      p->S > (1 << 20) || p->T > (1 << 24))
    return TA_ERR_UNSUPPORTED;
  return TA_OK;
}

// Sizes that the choice takes: a row's masses, and the queries of a key head,
// stand in shared memory; sequences and (row, key head) items are grid dimensions.
bool select_fits(const ta_cache_params* p) {
  return p->max_pages <= ta::kMaxSelectPages && p->H / p->Hkv <= 128 && p->S <= 65535 &&
         (int64_t)p->T * p->Hkv <= 0x7fffffff;
}
// The choice's scratch (none where it refuses the sizes): logits; and where rows
// may share their means, split means, their norms and scales, the queries'
// norms, the rows, and the list of items to do again.
size_t select_bytes(const ta_cache_params* p) {
  if (p->n_select <= 0 || !select_fits(p)) return 0;
  const size_t pitch = (size_t)ta::select_pitch(p->max_pages), T = (size_t)p->T + (p->T & 1);
  const size_t logits = pitch * p->H * 8 * ta::select_rows(p->H, p->T, p->max_pages);
  if (!ta::rows_share_means(p->T, p->S)) return logits;
  return logits + pitch * p->S * p->Hkv * (4 * p->d + 8) + T * p->H * 4 + (T + 2) * 8 + (size_t)p->T * p->Hkv * 8;
}
// Sparse attention's: parts of cut tiles, joint page lists and their lengths,
// the rows' flags.
size_t sparse_bytes(const ta_cache_params* p) {
  if (p->n_select <= 0) return 0;
  const int rows = ta::tile_rows(p->H / p->Hkv, p->T, p->S, p->max_pages);
  if (!rows) return 0;
  const size_t items = (size_t)ta::tile_count(rows, p->T, p->S) * p->Hkv;
  return ta::tile_part_bytes(items) + items * ((size_t)rows * p->n_select * 8 + 4) +
         ((size_t)p->T + 1 + ta::kMaxTileParts) * 4;
}
size_t scratch_bytes(const ta_cache_params* p) {
  const size_t a = select_bytes(p), b = sparse_bytes(p);
  return a > b ? a : b;
}

ta_status check_ws(const void* ws, size_t have, size_t need) {
  if (!aligned(ws, 256)) return TA_ERR_INVALID_ARG;
  return have < need ? TA_ERR_WORKSPACE : TA_OK;
}

// Strides of a bf16 [rows, heads, d] operand: 16-byte rows.
bool rows_ok(const void* ptr, int64_t st, int64_t sh) {
  return aligned(ptr, 16) && st % 8 == 0 && sh % 8 == 0;
}

// The cache's code strides, in elements of `esz` bytes (a dimension of size 1
// has no stride to speak of).
ta_status check_cache(const ta_cache_params* p, const ta_cache* c, bool kv, bool mean) {
  if (!c) return TA_ERR_INVALID_ARG;
  if (mean && !aligned(c->k_mean, 16)) return TA_ERR_INVALID_ARG;
  if (!kv) return TA_OK;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return TA_ERR_INVALID_ARG;
  const int esz = p->format == TA_CACHE_FP8 ? 1 : 2;
  if (esz == 1 && (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))) return TA_ERR_INVALID_ARG;
  if (p->stride_slot < p->d || (p->stride_slot * esz) % 16) return TA_ERR_INVALID_ARG;
  if (p->Hkv > 1 && (p->stride_head < p->d || (p->stride_head * esz) % 16)) return TA_ERR_INVALID_ARG;
  if (p->n_pages > 1 && (p->stride_page < p->d || (p->stride_page * esz) % 16))
    return TA_ERR_INVALID_ARG;
  const int64_t most = (int64_t)1 << 39;     // TMA strides are below 2^40 bytes
  if (p->stride_slot >= most || p->stride_head >= most || p->stride_page >= most)
    return TA_ERR_UNSUPPORTED;
  return TA_OK;
}

ta_status check_index(const ta_cache_params* p, const int32_t* cu, const int32_t* lens,
                      const int32_t* table) {
  if (!aligned(lens, 4) || !aligned(table, 4) || (cu && !aligned(cu, 4))) return TA_ERR_INVALID_ARG;
  if (p->stride_table < p->max_pages && p->S > 1) return TA_ERR_INVALID_ARG;
  if (!cu && p->T != p->S) return TA_ERR_INVALID_ARG;
  return TA_OK;
}

void fill(const ta_cache_params* p, const ta_cache* c, const int32_t* cu, const int32_t* lens,
          const int32_t* table, void* ws, CacheArgs& a) {
  a = CacheArgs{};
  a.n_pages = p->n_pages;
  a.page_size = p->page_size;
  a.ps_log2 = p->page_size == 16 ? 4 : p->page_size == 32 ? 5 : p->page_size == 64 ? 6 : 7;
  a.H = p->H;
  a.Hkv = p->Hkv;
  a.G = p->H / p->Hkv;
  a.d = p->d;
  a.fp8 = p->format == TA_CACHE_FP8;
  a.S = p->S;
  a.T = p->T;
  a.max_pages = p->max_pages;
  a.n_select = p->n_select;
  a.n_first = p->n_first;
  a.n_recent = p->n_recent;
  a.rot_dim = p->rot_dim;
  a.rot_interleaved = p->rot_interleaved;
  a.rot_rows = p->rot_rows;
  a.scale = p->softmax_scale > 0.0f ? (double)p->softmax_scale : 1.0 / std::sqrt((double)p->d);
  a.scale_log2 = (float)(a.scale * 1.4426950408889634);
  a.s_page = p->stride_page;
  a.s_head = p->stride_head;
  a.s_slot = p->stride_slot;
  a.s_table = p->stride_table;
  a.sk_t = p->stride_k_t;
  a.sk_h = p->stride_k_h;
  a.sv_t = p->stride_v_t;
  a.sv_h = p->stride_v_h;
  a.sq_t = p->stride_q_t;
  a.sq_h = p->stride_q_h;
  a.so_t = p->stride_o_t;
  a.so_h = p->stride_o_h;
  a.k = c->k;
  a.v = c->v;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.k_mean = c->k_mean;
  a.cu = cu;
  a.lens = lens;
  a.table = table;
  char* w = static_cast<char*>(ws);
  a.status = reinterpret_cast<int*>(w);
  a.counters = reinterpret_cast<int*>(w + ta::kWsCounters);
  a.part_ml = reinterpret_cast<float*>(w + ta::kWsPartML);
  a.part_o = reinterpret_cast<float*>(w + ta::kWsPartO);
  a.scratch = reinterpret_cast<double*>(w + ta::kWsScratch);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
                       cudaSuccess && q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<EncodeTiledFn>(f)
               : nullptr;
  }();
  return fn;
}

// Codes [n_pages, Hkv, page_size, d]: a box is one page of one head, 128 bytes
// of each row at most (64 for FP8 with d = 64), swizzled by the row's width.
// L2 fetches no more than a row at a time: behind it, in token-major pages,
// stands another head's, which comes too early for the block that wants it
// (551 MB of 128-byte rows: 106 us, with 256 bytes at a time 132; whole rows of
// 256 bytes gain by it, 107 us against 113 for 673 MB).
bool make_cache_map(CUtensorMap* m, const ta_cache_params* p, void* base) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const bool fp8 = p->format == TA_CACHE_FP8;
  const int esz = fp8 ? 1 : 2;
  const int box_bytes = p->d * esz < 128 ? 64 : 128;
  const int64_t slot = p->stride_slot * esz;
  const int64_t head = p->Hkv > 1 ? p->stride_head * esz : slot;
  const int64_t page = p->n_pages > 1 ? p->stride_page * esz : slot;
  cuuint64_t dims[4] = {(cuuint64_t)p->d, (cuuint64_t)p->page_size, (cuuint64_t)p->Hkv, (cuuint64_t)p->n_pages};
  cuuint64_t strides[3] = {(cuuint64_t)slot, (cuuint64_t)head, (cuuint64_t)page};
  cuuint32_t box[4] = {(cuuint32_t)(box_bytes / esz), (cuuint32_t)p->page_size, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            p->d * esz < 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

ta_status attend(const ta_cache_params* p, const ta_cache* cache, const void* Q, const int32_t* sel,
                 const int32_t* cu, const int32_t* lens, const int32_t* table, void* O, float* lse,
                 void* ws, size_t ws_bytes, void* stream, bool sparse) {
  ta_status st = check_cache(p, cache, true, false);
  if (st != TA_OK) return st;
  if ((st = check_index(p, cu, lens, table)) != TA_OK) return st;
  if (!rows_ok(Q, p->stride_q_t, p->stride_q_h) || !rows_ok(O, p->stride_o_t, p->stride_o_h) ||
      (lse && !aligned(lse, 4)))
    return TA_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, ta::kWsScratch + (sparse ? sparse_bytes(p) : 0))) != TA_OK) return st;
  if (sparse && O == Q) return TA_ERR_INVALID_ARG;   // (a row may be done again from its queries)
  CacheArgs a;
  fill(p, cache, cu, lens, table, ws, a);
  a.q = static_cast<const __nv_bfloat16*>(Q);
  a.o = static_cast<__nv_bfloat16*>(O);
  a.lse = lse;
  a.sel = const_cast<int32_t*>(sel);
  CUtensorMap mk, mv;
  if (!make_cache_map(&mk, p, cache->k) || !make_cache_map(&mv, p, cache->v)) return TA_ERR_CUDA;
  return ta::launch_cache_attn(a, mk, mv, sparse, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? TA_OK
             : TA_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t tiered_attn_cache_workspace_bytes(const ta_cache_params* p) {
  if (validate(p) != TA_OK) return 0;
  return (ta::kWsScratch + scratch_bytes(p) + 255) / 256 * 256;
}

ta_status tiered_attn_cache_init(void* ws, size_t ws_bytes, void* stream) {
  const ta_status st = check_ws(ws, ws_bytes, ta::kWsScratch);
  if (st != TA_OK) return st;
  // what later calls rely on being zero; partial results and scratch are
  // written before they are read
  return cudaMemsetAsync(ws, 0, ta::kWsPartML, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? TA_OK
             : TA_ERR_CUDA;
}

ta_status tiered_attn_cache_append(const ta_cache_params* p, const ta_cache* cache, const void* K_new,
                                   const void* V_new, const void* Q, void* Q_out, const float* cos,
                                   const float* sin, const int32_t* pos, const int32_t* cu,
                                   const int32_t* lens, const int32_t* table, void* ws,
                                   size_t ws_bytes, void* stream) {
  ta_status st = validate(p);
  if (st != TA_OK) return st;
  if ((st = check_cache(p, cache, true, cache && cache->k_mean)) != TA_OK) return st;
  if ((st = check_index(p, cu, lens, table)) != TA_OK) return st;
  if (!rows_ok(K_new, p->stride_k_t, p->stride_k_h) || !rows_ok(V_new, p->stride_v_t, p->stride_v_h))
    return TA_ERR_INVALID_ARG;
  if (Q && (!rows_ok(Q, p->stride_q_t, p->stride_q_h) || !rows_ok(Q_out, p->stride_o_t, p->stride_o_h)))
    return TA_ERR_INVALID_ARG;
  if (p->rot_dim && (!aligned(cos, 16) || !aligned(sin, 16))) return TA_ERR_INVALID_ARG;
  if (pos && !aligned(pos, 4)) return TA_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, ta::kWsScratch)) != TA_OK) return st;
  CacheArgs a;
  fill(p, cache, cu, lens, table, ws, a);
  a.k_new = static_cast<const __nv_bfloat16*>(K_new);
  a.v_new = static_cast<const __nv_bfloat16*>(V_new);
  a.q = static_cast<const __nv_bfloat16*>(Q);
  a.o = static_cast<__nv_bfloat16*>(Q_out);
  a.cos = cos;
  a.sin = sin;
  a.pos = pos;
  return ta::launch_cache_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? TA_OK
                                                                                       : TA_ERR_CUDA;
}

ta_status tiered_attn_cache_decode(const ta_cache_params* p, const ta_cache* cache, const void* Q,
                                   const int32_t* lens, const int32_t* table, void* O, float* lse,
                                   void* ws, size_t ws_bytes, void* stream) {
  ta_status st = validate(p);
  if (st != TA_OK) return st;
  // the kernel keeps a prefix over the sequences in shared memory, in 31 bits
  const int64_t units = ((int64_t)p->max_pages * p->page_size + 127) / 128;
  if (p->S > ta::kMaxDecodeSeqs || p->S * units > 0x7fffffff) return TA_ERR_UNSUPPORTED;
  return attend(p, cache, Q, nullptr, nullptr, lens, table, O, lse, ws, ws_bytes, stream, false);
}

ta_status tiered_attn_cache_select(const ta_cache_params* p, const ta_cache* cache, const void* Q,
                                   const int32_t* cu, const int32_t* lens, const int32_t* table,
                                   int32_t* sel, void* ws, size_t ws_bytes, void* stream) {
  ta_status st = validate(p);
  if (st != TA_OK) return st;
  if (p->n_select < 1) return TA_ERR_INVALID_ARG;
  if (!select_fits(p)) return TA_ERR_UNSUPPORTED;
  if ((st = check_cache(p, cache, false, true)) != TA_OK) return st;
  if ((st = check_index(p, cu, lens, table)) != TA_OK) return st;
  if (!rows_ok(Q, p->stride_q_t, p->stride_q_h) || !aligned(sel, 4)) return TA_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, ta::kWsScratch + select_bytes(p))) != TA_OK) return st;
  CacheArgs a;
  fill(p, cache, cu, lens, table, ws, a);
  a.q = static_cast<const __nv_bfloat16*>(Q);
  a.sel = sel;
  return ta::launch_cache_select(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? TA_OK
                                                                                       : TA_ERR_CUDA;
}

ta_status tiered_attn_cache_sparse(const ta_cache_params* p, const ta_cache* cache, const void* Q,
                                   const int32_t* sel, const int32_t* cu, const int32_t* lens,
                                   const int32_t* table, void* O, float* lse, void* ws,
                                   size_t ws_bytes, void* stream) {
  ta_status st = validate(p);
  if (st != TA_OK) return st;
  if (p->n_select < 1 || !aligned(sel, 4)) return TA_ERR_INVALID_ARG;
  return attend(p, cache, Q, sel, cu, lens, table, O, lse, ws, ws_bytes, stream, true);
}

}  // extern "C"
