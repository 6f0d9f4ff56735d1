// Paged key and value caches held in 4 bits, and the conversions their kernels share.
//
// Format: blocks of 16 elements of one row share a scale s, a multiple of an e4m3 number, and every
// element is one of the 16 e2m1 values {0, 0.5, 1, 1.5, 2, 3, 4, 6} with a sign, times s:
//   s_b = e4m3(max_i |x_i| / (6 g)),   code_i = e2m1(x_i / (s_b g)),   x_i ~ code_i s_b g
// with g one fp32 number per tensor (k_scale, v_scale), both conversions to nearest, ties to even.
// A row of d elements takes d/2 + d/16 bytes (4.5 bits an element).
//
// A pool holds pages [num_pages][H_kv][2][page_size * 9 d / 16]: the slab of one page, head and side
// (0 keys, 1 values) is page_size code rows of d/2 bytes, then page_size scale rows of d/16 bytes, so a
// page's slab is one contiguous piece and its rows are 16-byte (codes) and 4- or 8-byte (scales) aligned.
// Within a code row, byte (d/8) c + 2 j + i holds elements 16 j + 4 c + 2 i (low nibble) and the next
// one (high nibble), c < 4, j < d/16, i < 2: chunk c of a row is what lane c of a quad needs of it for
// every 16-element step of a matrix product, so fragments are read in whole 8- or 16-byte words.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace misa {

// Pages of one pool and the tables [sequences][max_pages] through which sequences own them.
struct RowPages {
  uint8_t* base;
  const int32_t* table;
  int64_t num_pages;
  int64_t max_pages;
  int page_size;
};

struct Kv4Pool : RowPages {
  int Hkv;
  int d;
  __host__ __device__ int64_t slab_bytes() const { return (int64_t)page_size * (9 * d / 16); }
  __host__ __device__ int64_t page_bytes() const { return slab_bytes() * 2 * Hkv; }
  __host__ __device__ int64_t scales_at() const { return (int64_t)page_size * (d / 2); }
};

// Physical page of logical row s of sequence t, or -1 when the table does not reach it or the page id
// is outside the pool (counted by the bounds-checked build where `count` is set).
__device__ __forceinline__ int64_t kv4_page(const RowPages& p, int64_t t, int64_t s, bool count) {
  if (s < 0) return -1;
  const uint32_t lp = (uint32_t)s / (uint32_t)p.page_size;
  if (lp >= p.max_pages) return -1;
  const int32_t pg = __ldg(p.table + t * p.max_pages + lp);
  if (pg < 0 || pg >= p.num_pages) {
    count_bad_id(kBadPage, count);
    return -1;
  }
  return pg;
}

// Four bytes of codes as four pairs of fp16 (low nibble in the low half); e2m1 is exact in fp16.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t x, uint32_t& h0, uint32_t& h1, uint32_t& h2, uint32_t& h3) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3)
      : "r"(x));
}

// Two e4m3 scales (low and high byte of x) as fp16; e4m3 is exact in fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}

// e2m1 codes of two values, `lo` in the low nibble; nearest, ties to even, magnitudes above 6 become 6.
__device__ __forceinline__ uint32_t float2_to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "cvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t float_to_e4m3(float x) {
  return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float e4m3_to_float(uint32_t x) {
  return __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_half2((uint16_t)x) & 0xffffu)));
}

}  // namespace misa
