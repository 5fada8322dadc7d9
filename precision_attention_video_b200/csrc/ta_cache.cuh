// ta_cache.cuh -- argument block, launchers and device helpers of the
// cached-attention kernels (append, decode, page choice, sparse attention).
#pragma once

#include <atomic>

#include "ta_common.cuh"
#include "tiered_attn_cache.h"

namespace ta {

// Fixed part of a cache workspace, the same whatever the parameters, so that
// calls with different ones can take turns on a workspace: the status word,
// one arrival counter and two partial results for each CTA of the attention
// grid.
constexpr int kMaxAttnCtas = 512;
constexpr int kMaxDecodeSeqs = 2048;              // rows of a decode (a prefix in shared memory)
constexpr int kMaxSelectPages = 16384;            // pages of a row that chooses (masses there)
constexpr int kMaxTileHeads = 16;                 // query heads of one CTA's item
constexpr size_t kWsCounters = 256;
constexpr size_t kWsPartML = kWsCounters + kMaxAttnCtas * 4;
constexpr size_t kWsPartO = kWsPartML + (size_t)kMaxAttnCtas * 2 * 2 * kMaxTileHeads * 4;
constexpr size_t kWsScratch = kWsPartO + (size_t)kMaxAttnCtas * 2 * kMaxTileHeads * 128 * 4;

struct CacheArgs {
  int n_pages, page_size, ps_log2;
  int H, Hkv, G, d, fp8;
  int S, T, max_pages;
  int n_select, n_first, n_recent;
  int rot_dim, rot_interleaved, rot_rows;
  float scale_log2;               // softmax scale * log2(e)
  double scale;                   // softmax scale (fp64, page choice)
  int64_t s_page, s_head, s_slot; // cache code strides (elements)
  int64_t s_table;
  int64_t sk_t, sk_h, sv_t, sv_h, sq_t, sq_h, so_t, so_h;
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  float* k_mean;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;               // O, or the rotated queries of an append
  float* lse;
  const float* cos;
  const float* sin;
  const int* pos;
  const int* cu;                  // null: one row for each sequence
  const int* lens;
  const int* table;
  int* sel;
  int* status;
  int* counters;
  float* part_ml;
  float* part_o;
  double* scratch;
  // page choice: rows that scratch has logits for, and those whose stand there
  int logit_rows, row0, row_n;
  // sparse attention of many rows (parts of scratch)
  int tile_rows;                  // rows that share their pages' loads
  int list_cap;                   // entries of a tile's page list
  int* row_flags;                 // [T] rows to do again on their own, [T]: any; null: all rows
  int* list_n;                    // [tile, Hkv] entries of the joint lists
  int* tile_arrived;              // [kMaxTileParts] parts of a cut tile that are done
  float* tile_parts;              // and their results
  int2* lists;                    // [tile, Hkv, list_cap] (page, bits of the rows that read it)
};

// Sparse attention takes rows of a sequence together where there are rows
// enough: up to 128 (row, query head) pairs to a tile, at most 32 rows (the bits
// of a list).  0: rows on their own.
inline int tile_rows(int G, int64_t T, int64_t S, int max_pages) {
  if (G > 64 || T < 4 * S || max_pages > kMaxSelectPages) return 0;
  return 128 / G < 32 ? 128 / G : 32;
}
constexpr int kMaxTileParts = 512;                // parts of cut tiles: 256 threads' 64 + 2 numbers each
// (a tile is cut into 8 parts at most)
inline size_t tile_part_bytes(int64_t items) {
  return (size_t)(items * 8 < kMaxTileParts ? items * 8 : kMaxTileParts) * (256 * 66 * 4);
}
inline int64_t tile_count(int rows, int64_t T, int64_t S) { return T / rows + S; }

// Doubles of a row of the choice's scratch: whole tiles of 128 pages.
__host__ __device__ inline int64_t select_pitch(int max_pages) { return ((int64_t)max_pages + 127) / 128 * 128; }
// Whether the logits of many rows may come from split means (given by cu).
inline bool rows_share_means(int64_t T, int64_t S) { return T >= 2 * S; }
// Rows that choose at a time: as many as have their logits in 4 GiB, so that a
// long prompt, or a table far wider than its sequences, does not ask for more.
// 32 query heads, 8 key heads, 1 GiB at a time, 4, and all at once: 8000 rows of
// tables of 8192 pages (16.9 GB) 3981, 2817 and 2682 us, 4680 rows (9.9 GB) 1640,
// 1374 and 1303, 32768 rows of 512 pages (4.3 GB) 1248, 1157 and 1188.
constexpr int64_t kMaxLogitBytes = (int64_t)1 << 32;
inline int select_rows(int H, int T, int max_pages) {
  const int64_t n = kMaxLogitBytes / (select_pitch(max_pages) * H * 8);
  return n < 1 ? 1 : n < T ? (int)n : T;
}

cudaError_t launch_cache_append(const CacheArgs& a, cudaStream_t s);
cudaError_t launch_cache_select(const CacheArgs& a, cudaStream_t s);
// `sparse`: over the lists in a.sel, else over whole sequences.
cudaError_t launch_cache_attn(const CacheArgs& a, const CUtensorMap& mk, const CUtensorMap& mv,
                              bool sparse, cudaStream_t s);

// The current device and its number of SMs, and a kernel's shared-memory limit
// raised once for each device: neither changes while the process lives.
struct OncePerDevice {
  std::atomic<unsigned long long> done{0};
  cudaError_t allow(const void* kernel, int dev, int bytes) {
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
  }
};
inline cudaError_t device_sms(int& dev, int& sms) {
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return e;
}

#ifdef __CUDACC__

__device__ __forceinline__ void report_bad_index(int* status) {
  if (atomicCAS(status + ST_CODE, 0, (int)TA_ERR_BAD_INDEX) == 0)
    status[ST_BLOCK] = (int)(blockIdx.x + gridDim.x * blockIdx.y);
}

// 8-byte asynchronous copy global -> shared.
__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Length of sequence s, clamped to what its table row can hold.
__device__ __forceinline__ int seq_len(const CacheArgs& a, int s) {
  const int n = a.lens[s];
  const int64_t most = (int64_t)a.max_pages << a.ps_log2;
  if (n < 0 || n > most) {
    report_bad_index(a.status);
    return n < 0 ? 0 : (int)most;
  }
  return n;
}

// Rows in use: everything from cu[S] on is padding.
__device__ __forceinline__ int rows_used(const CacheArgs& a) {
  if (!a.cu) return a.S;
  const int n = a.cu[a.S];
  return n < 0 ? 0 : (n > a.T ? a.T : n);
}

// Sequence of row t, and the row's position in it (-1 where the row has
// none: before the sequence's first position, or a malformed cu).
__device__ __forceinline__ int row_seq(const CacheArgs& a, int t) {
  if (!a.cu) return t;
  int lo = 0, hi = a.S - 1;       // largest s with cu[s] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ int row_pos(const CacheArgs& a, int t, int s) {
  const int n = seq_len(a, s);
  const int64_t back = a.cu ? (int64_t)a.cu[s + 1] - t : 1;
  const int64_t p = n - back;
  if (p >= 0 && p < n) return (int)p;
  if (a.cu) report_bad_index(a.status);   // (without cu, an empty sequence has no row)
  return -1;
}

// Physical page of entry e of sequence s; -1 (and the status) when the table
// holds a number outside the cache.
__device__ __forceinline__ int page_of(const CacheArgs& a, int s, int e) {
  const int pg = a.table[(int64_t)s * a.s_table + e];
  if (pg < 0 || pg >= a.n_pages) {
    report_bad_index(a.status);
    return -1;
  }
  return pg;
}

// Rows that a block takes together: up to tile_rows of one sequence.
struct RowTile {
  int s, t0, t1, t_end;
};
__device__ __forceinline__ RowTile row_tile(const CacheArgs& a, int tile, int tile_rows) {
  RowTile r;
  if (a.cu) {
    // tiles of sequence s start at cu[s] / tile_rows + s
    int lo = 0, hi = a.S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (max(a.cu[mid], 0) / tile_rows + mid <= tile) lo = mid; else hi = mid - 1;
    }
    r.s = lo;
    const int c0 = max(a.cu[lo], 0);
    r.t0 = c0 + (tile - (c0 / tile_rows + lo)) * tile_rows;
    r.t_end = min(a.cu[lo + 1], rows_used(a));
    r.t1 = min(r.t_end, r.t0 + tile_rows);
  } else {
    r.s = r.t0 = tile;
    r.t1 = r.t_end = tile + 1;
  }
  return r;
}

// 32 TMEM columns of this thread's lane at each of two addresses, waited for in
// the same statement: nothing can touch the registers before.
__device__ __forceinline__ void tmem_ld32x2(uint32_t ta, uint32_t tb, uint32_t (&a)[32], uint32_t (&b)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]),
        "=r"(a[7]), "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]),
        "=r"(a[14]), "=r"(a[15]), "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]),
        "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]), "=r"(a[24]), "=r"(a[25]),
        "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31]),
        "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]),
        "=r"(b[7]), "=r"(b[8]), "=r"(b[9]), "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]),
        "=r"(b[14]), "=r"(b[15]), "=r"(b[16]), "=r"(b[17]), "=r"(b[18]), "=r"(b[19]),
        "=r"(b[20]), "=r"(b[21]), "=r"(b[22]), "=r"(b[23]), "=r"(b[24]), "=r"(b[25]),
        "=r"(b[26]), "=r"(b[27]), "=r"(b[28]), "=r"(b[29]), "=r"(b[30]), "=r"(b[31])
      : "r"(ta), "r"(tb)
      : "memory");
}

#endif  // __CUDACC__

}  // namespace ta
