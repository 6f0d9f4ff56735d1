// C ABI of the attention beside the indexer: 4-bit caches, their attention and eviction, and prompt
// attention.  Argument checks and launches; declared and documented in include/misa.h.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "../../include/misa.h"
#include "kernels.cuh"

using misa::DType;
using misa::kMaxLen;
using misa::Kv4Pool;

namespace {

constexpr int kMaxPage = 1024;

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

misa_status launch_status() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MISA_OK : MISA_ERR_CUDA;
}

DType to_dtype(int dtype) { return dtype == MISA_F32 ? DType::F32 : DType::BF16; }

// The sizes of a 4-bit pool and its page tables.
misa_status check_kv4(int64_t num_pages, int page_size, int64_t max_pages, int H_kv, int d) {
  if (num_pages < 1 || page_size < 1 || max_pages < 1 || H_kv < 1) return MISA_ERR_INVALID_ARG;
  if (!misa::head_width(d)) return MISA_ERR_UNSUPPORTED;
  if (page_size % 16 != 0 || page_size > kMaxPage || H_kv > misa::kMaxKvHeads) return MISA_ERR_UNSUPPORTED;
  if (num_pages > INT32_MAX / page_size || max_pages > INT32_MAX) return MISA_ERR_UNSUPPORTED;
  return MISA_OK;
}

Kv4Pool to_pool(const void* pool, int64_t num_pages, int page_size, const int32_t* table, int64_t max_pages, int H_kv,
                int d) {
  Kv4Pool p;
  p.base = static_cast<uint8_t*>(const_cast<void*>(pool));
  p.table = table;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.page_size = page_size;
  p.Hkv = H_kv;
  p.d = d;
  return p;
}

bool positive(float x) { return x > 0.f && std::isfinite(x); }

// A cache's factor: far enough from the ends of fp32's range for a block's scale times it and its inverse.
bool factor(float x) { return x >= 0x1p-60f && x <= 0x1p60f; }

// Packed rows [rows][H][d] at stride ld elements that are read or written in 16-byte pieces.
misa_status check_rows(const void* p, int64_t ld, int H, int d, int dtype) {
  const int piece = dtype == MISA_F32 ? 4 : 8;
  if (!p || !at16(p) || ld < (int64_t)H * d || ld % piece != 0) return MISA_ERR_INVALID_ARG;
  return MISA_OK;
}

}  // namespace

extern "C" {

misa_status misa_kv4_append(const void* k, const void* v, int64_t ldk, int64_t ldv, int dtype, float k_scale,
                            float v_scale, void* pool, int64_t num_pages, int page_size, const int32_t* page_table,
                            int64_t max_pages, const int32_t* cu, const int32_t* start, int S, int rows, int H_kv,
                            int d, void* stream) {
  if (S < 0 || rows < 0) return MISA_ERR_INVALID_ARG;
  if (dtype != MISA_BF16 && dtype != MISA_F32) return MISA_ERR_UNSUPPORTED;
  misa_status st = check_kv4(num_pages, page_size, max_pages, H_kv, d);
  if (st != MISA_OK) return st;
  if (!factor(k_scale) || !factor(v_scale)) return MISA_ERR_INVALID_ARG;
  if ((int64_t)rows * H_kv > INT32_MAX) return MISA_ERR_UNSUPPORTED;
  if (S == 0 || rows == 0) return MISA_OK;
  if (!pool || !at16(pool) || !page_table || !cu || !start) return MISA_ERR_INVALID_ARG;
  st = check_rows(k, ldk, H_kv, d, dtype);
  if (st == MISA_OK) st = check_rows(v, ldv, H_kv, d, dtype);
  if (st != MISA_OK) return st;
  misa::launch_kv4_append(to_dtype(dtype), k, v, ldk, ldv,
                          to_pool(pool, num_pages, page_size, page_table, max_pages, H_kv, d), cu, start, S, rows,
                          k_scale, v_scale, static_cast<cudaStream_t>(stream));
  return launch_status();
}

misa_status misa_kv4_read(const void* pool, int64_t num_pages, int page_size, const int32_t* page_table,
                          int64_t max_pages, const int32_t* cu, const int32_t* start, int S, int rows, int H_kv, int d,
                          int dtype, float k_scale, float v_scale, void* k, void* v, void* stream) {
  if (S < 0 || rows < 0) return MISA_ERR_INVALID_ARG;
  if (dtype != MISA_BF16 && dtype != MISA_F32) return MISA_ERR_UNSUPPORTED;
  const misa_status st = check_kv4(num_pages, page_size, max_pages, H_kv, d);
  if (st != MISA_OK) return st;
  if (!factor(k_scale) || !factor(v_scale)) return MISA_ERR_INVALID_ARG;
  if ((int64_t)rows * H_kv > INT32_MAX) return MISA_ERR_UNSUPPORTED;
  if (S == 0 || rows == 0) return MISA_OK;
  if (!pool || !at16(pool) || !page_table || !cu || !start || !k || !v || !at16(k) || !at16(v))
    return MISA_ERR_INVALID_ARG;
  misa::launch_kv4_read(to_dtype(dtype), to_pool(pool, num_pages, page_size, page_table, max_pages, H_kv, d), cu,
                        start, S, rows, k_scale, v_scale, k, v, static_cast<cudaStream_t>(stream));
  return launch_status();
}

misa_status misa_kv4_attention(const void* q, const void* pool, int64_t num_pages, int page_size,
                               const int32_t* page_table, int64_t max_pages, const int32_t* n, const int32_t* idx,
                               int T, int L, int P, int H_q, int H_kv, int d, int dtype, float scale, float k_scale,
                               float v_scale, void* out, float* lse_opt, float* acc_opt, int64_t ld_acc, void* ws,
                               size_t ws_bytes, void* stream) {
  return misa_kv4_attention_cols(q, pool, num_pages, page_size, page_table, max_pages, n, idx, T, L, P, H_q, H_kv, d,
                                 dtype, scale, k_scale, v_scale, out, lse_opt, acc_opt, L, ld_acc, ws, ws_bytes, stream);
}

misa_status misa_kv4_attention_cols(const void* q, const void* pool, int64_t num_pages, int page_size,
                                    const int32_t* page_table, int64_t max_pages, const int32_t* n, const int32_t* idx,
                                    int T, int L, int P, int H_q, int H_kv, int d, int dtype, float scale,
                                    float k_scale, float v_scale, void* out, float* lse_opt, float* acc_opt,
                                    int acc_cols, int64_t ld_acc, void* ws, size_t ws_bytes, void* stream) {
  if (T < 0 || L < 1 || H_q < 1 || (idx && P < 1)) return MISA_ERR_INVALID_ARG;
  if (dtype != MISA_BF16 && dtype != MISA_F32) return MISA_ERR_UNSUPPORTED;
  const misa_status st = check_kv4(num_pages, page_size, max_pages, H_kv, d);
  if (st != MISA_OK) return st;
  if (H_q % H_kv != 0 || (int64_t)L > max_pages * page_size) return MISA_ERR_INVALID_ARG;
  if (L > kMaxLen || (idx && P > kMaxLen) || H_q > misa::kMaxQueryHeads) return MISA_ERR_UNSUPPORTED;
  if (!positive(scale) || !factor(k_scale) || !factor(v_scale)) return MISA_ERR_INVALID_ARG;
  if (acc_opt && (acc_cols < 1 || ld_acc < acc_cols)) return MISA_ERR_INVALID_ARG;
  if (T == 0) return MISA_OK;
  if (!q || !at16(q) || !pool || !at16(pool) || !page_table || !n || !out || !at16(out)) return MISA_ERR_INVALID_ARG;
  const int seen = idx ? P : L;
  if (!ws || ws_bytes < misa::kv4_attention_ws_bytes(T, seen, H_q, H_kv, d, acc_opt != nullptr) ||
      (reinterpret_cast<uintptr_t>(ws) & 255))
    return MISA_ERR_WORKSPACE;
  misa::launch_kv4_attention(to_dtype(dtype), q, to_pool(pool, num_pages, page_size, page_table, max_pages, H_kv, d), n,
                             idx, T, L, seen, H_q, scale, k_scale, v_scale, out, lse_opt, acc_opt, acc_cols, ld_acc,
                             ws, static_cast<cudaStream_t>(stream));
  return launch_status();
}

misa_status misa_evict_select(const float* acc, int64_t ld_acc, const int32_t* n, int T, int L, int keep, int sink,
                              int recent, int32_t* idx, int32_t* n_out, float* acc_out_opt, int64_t ld_out,
                              void* stream) {
  if (T < 0 || L < 1 || keep < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > keep || ld_acc < L)
    return MISA_ERR_INVALID_ARG;
  if (L > kMaxLen || keep > kMaxLen) return MISA_ERR_UNSUPPORTED;
  if (acc_out_opt && ld_out < keep) return MISA_ERR_INVALID_ARG;
  if (T == 0) return MISA_OK;
  if (!acc || !n || !idx || !n_out) return MISA_ERR_INVALID_ARG;
  if (acc_out_opt) {  // the kept weights are written while others are read
    const float *a0 = acc, *a1 = acc + (int64_t)(T - 1) * ld_acc + L, *b0 = acc_out_opt,
                *b1 = acc_out_opt + (int64_t)T * ld_out;
    if (a0 < b1 && b0 < a1) return MISA_ERR_INVALID_ARG;
  }
  // the lengths may be updated in place, but no row may write another row's
  if (n_out != n && n_out < n + T && n < n_out + T) return MISA_ERR_INVALID_ARG;
  misa::launch_evict_select(acc, ld_acc, n, T, L, keep, sink, recent, idx, n_out, acc_out_opt, ld_out,
                            static_cast<cudaStream_t>(stream));
  return launch_status();
}

misa_status misa_kv4_compact(void* pool, int64_t num_pages, int page_size, const int32_t* page_table,
                             int64_t max_pages, const int32_t* idx, int T, int keep, int H_kv, int d, void* ws,
                             size_t ws_bytes, void* stream) {
  if (T < 0 || keep < 1) return MISA_ERR_INVALID_ARG;
  const misa_status st = check_kv4(num_pages, page_size, max_pages, H_kv, d);
  if (st != MISA_OK) return st;
  if ((int64_t)keep > max_pages * page_size) return MISA_ERR_INVALID_ARG;
  if (keep > kMaxLen) return MISA_ERR_UNSUPPORTED;
  if (T == 0) return MISA_OK;
  if (!pool || !at16(pool) || !page_table || !idx) return MISA_ERR_INVALID_ARG;
  if (!ws || ws_bytes < misa::compact_ws_bytes(T, keep, 2 * H_kv, d / 2, d / 16) || (reinterpret_cast<uintptr_t>(ws) & 255))
    return MISA_ERR_WORKSPACE;
  const Kv4Pool p = to_pool(pool, num_pages, page_size, page_table, max_pages, H_kv, d);
  if (!misa::launch_compact_rows(p, 2 * H_kv, p.slab_bytes(), d / 2, d / 16, idx, T, keep, ws,
                                 static_cast<cudaStream_t>(stream)))
    return MISA_ERR_CUDA;
  return launch_status();
}

misa_status misa_keys_compact_paged(void* pool, int64_t num_pages, int page_size, const int32_t* page_table,
                                    int64_t max_pages, const int32_t* idx, int T, int keep, int d, int dtype, void* ws,
                                    size_t ws_bytes, void* stream) {
  if (T < 0 || keep < 1 || num_pages < 1 || page_size < 1 || max_pages < 1) return MISA_ERR_INVALID_ARG;
  if (dtype != MISA_BF16 && dtype != MISA_F32) return MISA_ERR_UNSUPPORTED;
  if (d != misa::kD) return MISA_ERR_UNSUPPORTED;
  if (num_pages > INT32_MAX / page_size || max_pages > INT32_MAX) return MISA_ERR_UNSUPPORTED;
  if ((int64_t)keep > max_pages * page_size) return MISA_ERR_INVALID_ARG;
  if (keep > kMaxLen) return MISA_ERR_UNSUPPORTED;
  if (T == 0) return MISA_OK;
  if (!pool || !at16(pool) || !page_table || !idx) return MISA_ERR_INVALID_ARG;
  const int rb = d * (dtype == MISA_F32 ? 4 : 2);
  if (!ws || ws_bytes < misa::compact_ws_bytes(T, keep, 1, rb, 0) || (reinterpret_cast<uintptr_t>(ws) & 255))
    return MISA_ERR_WORKSPACE;
  misa::RowPages p;
  p.base = static_cast<uint8_t*>(pool);
  p.table = page_table;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.page_size = page_size;
  if (!misa::launch_compact_rows(p, 1, (int64_t)page_size * rb, rb, 0, idx, T, keep, ws, static_cast<cudaStream_t>(stream)))
    return MISA_ERR_CUDA;
  return launch_status();
}

misa_status misa_prompt_attention(const void* q, const void* k, const void* v, int64_t ldq, int64_t ldk, int64_t ldv,
                                  const int32_t* cu_q, const int32_t* cu_k, int S, int Tq, int Tk, int H_q, int H_kv,
                                  int d, int dtype, float scale, void* out, float* lse_opt, void* ws, size_t ws_bytes,
                                  void* stream) {
  if (S < 0 || Tq < 0 || Tk < 0 || H_q < 1 || H_kv < 1) return MISA_ERR_INVALID_ARG;
  if (dtype != MISA_BF16) return MISA_ERR_UNSUPPORTED;
  if (!misa::head_width(d)) return MISA_ERR_UNSUPPORTED;
  if (H_q % H_kv != 0 || !positive(scale)) return MISA_ERR_INVALID_ARG;
  if (Tq > kMaxLen || Tk > kMaxLen || H_q > misa::kMaxPromptHeads) return MISA_ERR_UNSUPPORTED;
  if (S == 0 || Tq == 0) return MISA_OK;
  if (!cu_q || !cu_k || !out || !at16(out)) return MISA_ERR_INVALID_ARG;
  misa_status st = check_rows(q, ldq, H_q, d, dtype);
  if (st == MISA_OK && Tk > 0) st = check_rows(k, ldk, H_kv, d, dtype);
  if (st == MISA_OK && Tk > 0) st = check_rows(v, ldv, H_kv, d, dtype);
  if (st != MISA_OK) return st;
  const size_t need = misa::prompt_ws_bytes(S, Tq, Tk, H_q, d);
  if (need > 0 && (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255))) return MISA_ERR_WORKSPACE;
  if (!misa::launch_prompt_attention(q, k, v, ldq, ldk, ldv, cu_q, cu_k, S, Tq, Tk, H_q, H_kv, d, scale, out, lse_opt, ws,
                                     static_cast<cudaStream_t>(stream)))
    return MISA_ERR_UNSUPPORTED;
  return launch_status();
}

}  // extern "C"
