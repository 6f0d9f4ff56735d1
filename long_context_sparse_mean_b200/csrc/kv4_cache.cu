// The 4-bit caches' upkeep (format in kv4.cuh): rows written as they are computed, read back, and
// closed up after an eviction.
#include "kernels.cuh"
#include "kv4.cuh"

namespace misa {

namespace {

constexpr int64_t kCompactWsBytes = 32ll << 20;  // workspace of a compaction: stays in the L2 (126 MB)

// Sequence of packed row r: the last b with cu[b] <= r, or -1 when the row lies outside
// [cu[0], cu[S]).  Sequences without rows are passed over.
__device__ __forceinline__ int packed_seq(const int32_t* __restrict__ cu, int S, int r) {
  if (r < __ldg(cu) || r >= __ldg(cu + S)) return -1;
  int lo = 0, hi = S;  // cu[lo] <= r < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <DType DT>
__device__ __forceinline__ void load_block16(const void* base, int64_t at, float (&x)[16]) {
  if (DT == DType::BF16) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = __ldg(p + i);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[8 * i + 2 * e] = bf16_lo(w[e]);
        x[8 * i + 2 * e + 1] = bf16_hi(w[e]);
      }
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 u = __ldg(p + i);
      x[4 * i] = u.x;
      x[4 * i + 1] = u.y;
      x[4 * i + 2] = u.z;
      x[4 * i + 3] = u.w;
    }
  }
}

// One thread per 16-element block of (row, head, side).
template <DType DT>
__global__ void __launch_bounds__(256) kv4_append_kernel(const void* __restrict__ k, const void* __restrict__ v,
                                                         int64_t ldk, int64_t ldv, Kv4Pool pool,
                                                         const int32_t* __restrict__ cu,
                                                         const int32_t* __restrict__ start, int S, int rows, float kg,
                                                         float vg) {
  const int nb = pool.d / 16;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t per = (int64_t)pool.Hkv * 2 * nb;
  const int64_t r = i / per;
  if (r >= rows) return;
  const int u = (int)(i - r * per);
  const int b = u % nb, side = (u / nb) & 1, h = u / (2 * nb);
  const int seq = packed_seq(cu, S, (int)r);
  if (seq < 0) return;
  const int64_t s = (int64_t)__ldg(start + seq) + (r - __ldg(cu + seq));
  const int64_t pg = kv4_page(pool, seq, s, u == 0);
  if (pg < 0) return;
  float x[16];
  load_block16<DT>(side ? v : k, r * (side ? ldv : ldk) + (int64_t)h * pool.d + b * 16, x);
  const float g = side ? vg : kg;
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    x[e] = x[e] == x[e] ? x[e] : 0.f;  // NaN stores as 0
    top = fmaxf(top, fabsf(x[e]));
  }
  const uint32_t s8 = float_to_e4m3(top / (g * 6.0f));
  const float unit = e4m3_to_float(s8) * g;
  uint8_t* slab = pool.base + pg * pool.page_bytes() + (int64_t)(2 * h + side) * pool.slab_bytes();
  const int at = (int)(s % pool.page_size);
  uint8_t* row = slab + (int64_t)at * (pool.d / 2);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t code = 0;
    if (unit != 0.f)
      code = float2_to_e2m1x2(x[4 * c] / unit, x[4 * c + 1] / unit) |
             (float2_to_e2m1x2(x[4 * c + 2] / unit, x[4 * c + 3] / unit) << 8);
    *reinterpret_cast<uint16_t*>(row + (pool.d / 8) * c + 2 * b) = (uint16_t)code;
  }
  slab[pool.scales_at() + (int64_t)at * nb + b] = (uint8_t)s8;
}

// One thread per 16-element block of (row, head, side).
template <DType DT>
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4Pool pool, const int32_t* __restrict__ cu,
                                                       const int32_t* __restrict__ start, int S, int rows, float kg,
                                                       float vg, void* __restrict__ k, void* __restrict__ v) {
  const int nb = pool.d / 16;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t per = (int64_t)pool.Hkv * 2 * nb;
  const int64_t r = i / per;
  if (r >= rows) return;
  const int u = (int)(i - r * per);
  const int b = u % nb, side = (u / nb) & 1, h = u / (2 * nb);
  const int seq = packed_seq(cu, S, (int)r);
  if (seq < 0) return;
  const int64_t s = (int64_t)__ldg(start + seq) + (r - __ldg(cu + seq));
  const int64_t pg = kv4_page(pool, seq, s, u == 0);
  float x[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = 0.f;
  if (pg >= 0) {
    const uint8_t* slab = pool.base + pg * pool.page_bytes() + (int64_t)(2 * h + side) * pool.slab_bytes();
    const int at = (int)(s % pool.page_size);
    const uint8_t* row = slab + (int64_t)at * (pool.d / 2);
    const float sc = e4m3_to_float(slab[pool.scales_at() + (int64_t)at * nb + b]), g = side ? vg : kg;
    uint32_t w[2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
      w[c] = (uint32_t)*reinterpret_cast<const uint16_t*>(row + (pool.d / 8) * (2 * c) + 2 * b) |
             ((uint32_t)*reinterpret_cast<const uint16_t*>(row + (pool.d / 8) * (2 * c + 1) + 2 * b) << 16);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t y[4];
      e2m1x8_to_half2(w[c], y[0], y[1], y[2], y[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y[e]));
        x[8 * c + 2 * e] = f.x * sc * g;
        x[8 * c + 2 * e + 1] = f.y * sc * g;
      }
    }
  }
  const int64_t at = ((int64_t)r * pool.Hkv + h) * pool.d + b * 16;
  if (DT == DType::BF16) {
    uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(side ? v : k) + at);
    uint32_t y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      y[e] = *reinterpret_cast<const uint32_t*>(&p);
    }
    o[0] = make_uint4(y[0], y[1], y[2], y[3]);
    o[1] = make_uint4(y[4], y[5], y[6], y[7]);
  } else {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(side ? v : k) + at);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
  }
}

// Rows [j0, j0 + C) of every sequence's kept list, between the pool and the workspace
// [T][C][slabs][row bytes].  Moving a chunk takes two launches: the first copies rows idx[t, j] out, the
// second writes them to rows j.  idx is ascending, so idx[t, j] >= j: a chunk's writes land on rows
// below every row that a later chunk reads, and every earlier chunk has been read already.  Rows that
// stay where they are (idx[t, j] == j) are not touched.
// A unit is 16 bytes of a code row, or the whole scale row (sb bytes, 4 or 8; 0: the pool has none).
template <bool OUT>
__global__ void __launch_bounds__(256) compact_rows_kernel(RowPages pages, int slabs, int64_t slab_bytes,
                                                           int rb, int sb, const int32_t* __restrict__ idx, int T,
                                                           int keep, int j0, int C, uint8_t* __restrict__ ws) {
  const int units = rb / 16 + (sb ? 1 : 0);
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t per = (int64_t)slabs * C * units;
  const int64_t t = i / per;
  if (t >= T) return;
  int64_t x = i - t * per;
  const int slab = (int)(x / ((int64_t)C * units));
  x -= (int64_t)slab * C * units;
  const int jj = (int)(x / units), u = (int)(x - (int64_t)jj * units);
  const int j = j0 + jj;
  if (j >= keep) return;
  const int src = __ldg(idx + t * keep + j);
  if (src < 0 || src == j) return;
  // a row whose source or own place the table does not hold stays as it is
  const bool count = OUT && slab == 0 && u == 0;
  const int64_t pj = kv4_page(pages, t, j, false), ps = kv4_page(pages, t, src, count);
  if (pj < 0 || ps < 0) return;
  const int64_t s = OUT ? src : j, pg = OUT ? ps : pj;
  const int at = (int)(s % pages.page_size);
  uint8_t* base = pages.base + (pg * slabs + slab) * slab_bytes;
  uint8_t* w = ws + (t * slabs + slab) * C * (int64_t)(rb + sb);
  if (u * 16 < rb) {
    uint4* a = reinterpret_cast<uint4*>(base + (int64_t)at * rb + u * 16);
    uint4* b = reinterpret_cast<uint4*>(w + (int64_t)jj * rb + u * 16);
    if (OUT) *b = *a;
    else *a = *b;
  } else {
    uint8_t* a = base + (int64_t)pages.page_size * rb + (int64_t)at * sb;
    uint8_t* b = w + (int64_t)C * rb + (int64_t)jj * sb;
    if (sb == 8) {
      if (OUT) *reinterpret_cast<uint2*>(b) = *reinterpret_cast<const uint2*>(a);
      else *reinterpret_cast<uint2*>(a) = *reinterpret_cast<const uint2*>(b);
    } else {
      if (OUT) *reinterpret_cast<uint32_t*>(b) = *reinterpret_cast<const uint32_t*>(a);
      else *reinterpret_cast<uint32_t*>(a) = *reinterpret_cast<const uint32_t*>(b);
    }
  }
}

}  // namespace

void launch_kv4_append(DType dt, const void* k, const void* v, int64_t ldk, int64_t ldv, const Kv4Pool& pool,
                       const int32_t* cu, const int32_t* start, int S, int rows, float kg, float vg, cudaStream_t s) {
  if (S <= 0 || rows <= 0) return;
  const int64_t threads = (int64_t)rows * pool.Hkv * 2 * (pool.d / 16);
  const unsigned grid = (unsigned)((threads + 255) / 256);
  if (dt == DType::BF16)
    kv4_append_kernel<DType::BF16><<<grid, 256, 0, s>>>(k, v, ldk, ldv, pool, cu, start, S, rows, kg, vg);
  else
    kv4_append_kernel<DType::F32><<<grid, 256, 0, s>>>(k, v, ldk, ldv, pool, cu, start, S, rows, kg, vg);
}

void launch_kv4_read(DType dt, const Kv4Pool& pool, const int32_t* cu, const int32_t* start, int S, int rows,
                     float kg, float vg, void* k, void* v, cudaStream_t s) {
  if (S <= 0 || rows <= 0) return;
  const int64_t threads = (int64_t)rows * pool.Hkv * 2 * (pool.d / 16);
  const unsigned grid = (unsigned)((threads + 255) / 256);
  if (dt == DType::BF16)
    kv4_read_kernel<DType::BF16><<<grid, 256, 0, s>>>(pool, cu, start, S, rows, kg, vg, k, v);
  else
    kv4_read_kernel<DType::F32><<<grid, 256, 0, s>>>(pool, cu, start, S, rows, kg, vg, k, v);
}

// Rows per chunk of a compaction: what fits the workspace piece (at least one row of every sequence).
int compact_chunk(int T, int keep, int64_t row_bytes) {
  const int64_t fit = kCompactWsBytes / (row_bytes * T) / 16 * 16;
  return (int)(fit < 16 ? 16 : (fit < keep ? fit : (keep + 15) / 16 * 16));
}

size_t compact_ws_bytes(int T, int keep, int64_t row_bytes) {
  return (size_t)T * compact_chunk(T, keep, row_bytes) * row_bytes;
}

void launch_compact_rows(const RowPages& pages, int slabs, int64_t slab_bytes, int rb, int sb, const int32_t* idx,
                         int T, int keep, void* ws, cudaStream_t s) {
  if (T <= 0 || keep <= 0) return;
  const int C = compact_chunk(T, keep, (int64_t)slabs * (rb + sb));
  const int units = rb / 16 + (sb ? 1 : 0);
  for (int j0 = 0; j0 < keep; j0 += C) {
    const int64_t threads = (int64_t)T * slabs * C * units;
    const unsigned grid = (unsigned)((threads + 255) / 256);
    compact_rows_kernel<true><<<grid, 256, 0, s>>>(pages, slabs, slab_bytes, rb, sb, idx, T, keep, j0, C,
                                                   static_cast<uint8_t*>(ws));
    compact_rows_kernel<false><<<grid, 256, 0, s>>>(pages, slabs, slab_bytes, rb, sb, idx, T, keep, j0, C,
                                                    static_cast<uint8_t*>(ws));
  }
}

MISA_BAD_ID_READER(read_and_clear_bad_ids_kv4_cache)

}  // namespace misa
