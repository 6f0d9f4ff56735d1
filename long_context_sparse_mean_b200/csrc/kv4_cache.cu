// The 4-bit caches' upkeep (format in kv4.cuh): rows written as they are computed, read back, and
// closed up after an eviction.
#include <algorithm>

#include "kernels.cuh"
#include "kv4.cuh"

namespace misa {

namespace {

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

// x / b to nearest for finite b away from the ends of fp32's range, given y = 1 / b to nearest (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990: the residual of the
// first quotient is exact in one fused multiply-add, and a second adds it in).  Quotients past 8 keep
// their sign and stay past 8, infinite x included, which is all that the conversion to e2m1 needs.
__device__ __forceinline__ float divide(float x, float b, float y) {
  const float q = fminf(fmaxf(x * y, -8.f), 8.f);
  return fmaf(fmaf(-q, b, x), y, q);
}

// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Both kernels: four threads a row of a head and side; thread c has the elements 16 j + 4 c .. + 3 of every
// block j, which are chunk c of the code row, so codes move in whole 16-byte (d = 64: 8-byte) words and
// the elements in 8- or 16-byte pieces of which four threads cover a full 32- or 64-byte stretch.  What
// bounds them is HBM: every element is read or written once in its own type, every code once.  13.3K rows of 8
// heads of 128 in bf16: append 24.6 us, 2.8 TB/s (conversions and the five operations of a
// quotient for every element; with the scales worked out by all four threads 31.3), read back 15.2 us, 4.6 TB/s.
template <int D, DType DT>
__global__ void __launch_bounds__(256) kv4_append_kernel(const void* __restrict__ k, const void* __restrict__ v,
                                                         int64_t ldk, int64_t ldv, Kv4Pool pool,
                                                         const int32_t* __restrict__ cu,
                                                         const int32_t* __restrict__ start, int S, int rows, float kg,
                                                         float vg) {
  constexpr int NB = D / 16;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int c = (int)(i & 3), sides = 2 * pool.Hkv;
  const bool in = (i >> 2) < (int64_t)rows * sides;  // whole groups of four threads alike; they exchange maxima below
  const uint32_t u = (uint32_t)(i >> 2);             // rows and heads are bounded: 32 bits hold it
  const int64_t r = u / (uint32_t)sides;
  const int sl = (int)(u - (uint32_t)r * sides), h = sl >> 1, side = sl & 1;
  float x[NB][4];
  if (in) {
    const int64_t at = r * (side ? ldv : ldk) + (int64_t)h * D + 4 * c;
    const void* base = side ? v : k;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if (DT == DType::BF16) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + at + 16 * j));
        x[j][0] = bf16_lo(w.x);
        x[j][1] = bf16_hi(w.x);
        x[j][2] = bf16_lo(w.y);
        x[j][3] = bf16_hi(w.y);
      } else {
        const float4 w = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + at + 16 * j));
        x[j][0] = w.x;
        x[j][1] = w.y;
        x[j][2] = w.z;
        x[j][3] = w.w;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NB; ++j) x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.f;
  }
  const int seq = in ? packed_seq(cu, S, (int)r) : -1;
  int64_t s = 0, pg = -1;
  if (seq >= 0) {
    s = (int64_t)__ldg(start + seq) + (r - __ldg(cu + seq));
    pg = kv4_page(pool, seq, s, sl == 0 && c == 0);
  }
  // The four threads find the largest elements of their NB blocks together, each ending up with those of its own
  // NB / 4 blocks, whose scales and inverses it works out for all four (a division and a reciprocal to nearest
  // are as long as all the rest of a block).
  constexpr int OWN = NB / 4;
  const float g = side ? vg : kg, g6 = g * 6.0f;
  float top[OWN];
  auto tops = [&] {
    float m[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
      m[j] = max_nan(max_nan(fabsf(x[j][0]), fabsf(x[j][1])), max_nan(fabsf(x[j][2]), fabsf(x[j][3])));
#pragma unroll
    for (int j = 0; j < NB / 2; ++j) {
      const float got = __shfl_xor_sync(0xffffffffu, c & 2 ? m[j] : m[j + NB / 2], 2);
      m[j] = max_nan(c & 2 ? m[j + NB / 2] : m[j], got);
    }
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
      const float got = __shfl_xor_sync(0xffffffffu, c & 1 ? m[j] : m[j + OWN], 1);
      top[j] = max_nan(c & 1 ? m[j + OWN] : m[j], got);
    }
  };
  tops();
  bool nan = false;
#pragma unroll
  for (int j = 0; j < OWN; ++j) nan |= top[j] != top[j];
  if (__any_sync(0xffffffffu, nan)) {  // NaN stores as 0
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[j][e] = x[j][e] == x[j][e] ? x[j][e] : 0.f;
    tops();
  }
  float unit[OWN], inv[OWN];
  uint32_t s8 = 0;
#pragma unroll
  for (int j = 0; j < OWN; ++j) {
    const uint32_t e = float_to_e4m3(top[j] / g6);
    unit[j] = e4m3_to_float(e) * g;
    inv[j] = unit[j] == 0.f ? 0.f : __frcp_rn(unit[j]);  // with both 0 every quotient is 0, of x's sign
    s8 |= e << (8 * j);
  }
  uint32_t code[NB / 2], scale[NB / 4];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const float u = __shfl_sync(0xffffffffu, unit[j % OWN], j / OWN, 4);
    const float y = __shfl_sync(0xffffffffu, inv[j % OWN], j / OWN, 4);
    const uint32_t w = float2_to_e2m1x2(divide(x[j][0], u, y), divide(x[j][1], u, y)) |
                       (float2_to_e2m1x2(divide(x[j][2], u, y), divide(x[j][3], u, y)) << 8);
    code[j / 2] = j & 1 ? code[j / 2] | (w << 16) : w;
  }
#pragma unroll
  for (int j = 0; j < NB / 4; ++j) {
    scale[j] = 0;
#pragma unroll
    for (int k = 0; k < 4 / OWN; ++k)
      scale[j] |= __shfl_sync(0xffffffffu, s8, j * (4 / OWN) + k, 4) << (8 * OWN * k);
  }
  if (pg < 0) return;
  uint8_t* slab = pool.base + pg * pool.page_bytes() + (int64_t)sl * pool.slab_bytes();
  const int at = (int)((uint32_t)s % (uint32_t)pool.page_size);
  uint8_t* row = slab + (int64_t)at * (D / 2) + c * (D / 8);
  uint8_t* sc = slab + pool.scales_at() + (int64_t)at * NB;
  if constexpr (D == 128) {
    *reinterpret_cast<uint4*>(row) = make_uint4(code[0], code[1], code[2], code[3]);
    if (c == 0) *reinterpret_cast<uint2*>(sc) = make_uint2(scale[0], scale[1]);
  } else {
    *reinterpret_cast<uint2*>(row) = make_uint2(code[0], code[1]);
    if (c == 0) *reinterpret_cast<uint32_t*>(sc) = scale[0];
  }
}

template <int D, DType DT>
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4Pool pool, const int32_t* __restrict__ cu,
                                                       const int32_t* __restrict__ start, int S, int rows, float kg,
                                                       float vg, void* __restrict__ k, void* __restrict__ v) {
  constexpr int NB = D / 16;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int c = (int)(i & 3), sides = 2 * pool.Hkv;
  if ((i >> 2) >= (int64_t)rows * sides) return;
  const uint32_t u = (uint32_t)(i >> 2);
  const int64_t r = u / (uint32_t)sides;
  const int sl = (int)(u - (uint32_t)r * sides), h = sl >> 1, side = sl & 1;
  const int seq = packed_seq(cu, S, (int)r);
  if (seq < 0) return;
  const int64_t s = (int64_t)__ldg(start + seq) + (r - __ldg(cu + seq));
  const int64_t pg = kv4_page(pool, seq, s, sl == 0 && c == 0);
  uint32_t code[NB / 2], scale[NB / 4];
#pragma unroll
  for (int j = 0; j < NB / 2; ++j) code[j] = 0u;
#pragma unroll
  for (int j = 0; j < NB / 4; ++j) scale[j] = 0u;
  if (pg >= 0) {
    const uint8_t* slab = pool.base + pg * pool.page_bytes() + (int64_t)sl * pool.slab_bytes();
    const int at = (int)((uint32_t)s % (uint32_t)pool.page_size);
    const uint8_t* row = slab + (int64_t)at * (D / 2) + c * (D / 8);
    const uint8_t* sc = slab + pool.scales_at() + (int64_t)at * NB;
    if constexpr (D == 128) {
      const uint4 w = *reinterpret_cast<const uint4*>(row);
      const uint2 e = *reinterpret_cast<const uint2*>(sc);
      code[0] = w.x, code[1] = w.y, code[2] = w.z, code[3] = w.w;
      scale[0] = e.x, scale[1] = e.y;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(row);
      code[0] = w.x, code[1] = w.y;
      scale[0] = *reinterpret_cast<const uint32_t*>(sc);
    }
  }
  const float g = side ? vg : kg;
  const int64_t at = (r * pool.Hkv + h) * D + 4 * c;
#pragma unroll
  for (int w = 0; w < NB / 2; ++w) {
    uint32_t y[4];
    e2m1x8_to_half2(code[w], y[0], y[1], y[2], y[3]);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int j = 2 * w + b;
      const float sc = e4m3_to_float((scale[j / 4] >> (8 * (j & 3))) & 255u);
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&y[2 * b]));
      const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&y[2 * b + 1]));
      const float x0 = p.x * sc * g, x1 = p.y * sc * g, x2 = q.x * sc * g, x3 = q.y * sc * g;
      if (DT == DType::BF16) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x0, x1), hi = __floats2bfloat162_rn(x2, x3);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(side ? v : k) + at + 16 * j) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(side ? v : k) + at + 16 * j) = make_float4(x0, x1, x2, x3);
      }
    }
  }
}

// Closes up caches in place: row idx[t, j] of sequence t moves to row j, for all j.  A CTA takes a segment
// of R rows j of one sequence and a group of slabs: it reads their sources into shared memory, marks its
// segment as read, waits until every segment whose sources lie where it is going to write has been
// marked, and writes.  idx is ascending, so idx[t, j] >= j: a segment's own place is read by itself and by
// segments before it alone; they are found by searching idx for the ends of the place while the copies are
// under way.  Segments are handed out in order by a counter of each sequence and group, not by block index, so
// that those before a CTA's own are with CTAs that run already, whatever order CTAs start in, and a segment
// is marked before its CTA waits for any.  (In the usual case of a part kept, rows come from far behind their
// new place, and the segments waited for finished long ago.)  A short list is one segment and needs no marks.
// Rows that stay where they are are passed over, and so are rows whose own or source page is not in the
// pool.  Bound by HBM: rows are read and written once, but rows of 64 and 8 bytes from here and there fetch up
// to twice their size.  16 caches of up to 32768 tokens thinned to 8192 (8 heads of 128): 65 us for 85 MB moved,
// with 160 MB read (63 with segments by block index); the indexer's bf16 keys beside them 17 us.  In chunks through workspace: 259 us.  (36 KB of
// rows in CTAs of 256 threads: one cache of 128K tokens 8 us faster, this batch 2 us slower.)
// Waits are bounded (1 s); a segment whose wait runs out is not written and a status word is set.
constexpr int kSeg = 64;                // fewest rows of a segment where there are several
constexpr int kGpuSms = 148;
constexpr int kGroupBytes = 72 * 1024;  // its rows in shared memory: three CTAs an SM
constexpr int kOneSeg = 512;            // longest list taken as one segment,
constexpr int kOneSegBytes = 160 * 1024;  // where a slab's rows of it fit here
constexpr int kFewCtas = 96;
constexpr int kCompactThreads = 512;
constexpr uint64_t kWaitLimitNs = 1000000000ull;

__device__ int g_compact_status = 0;

__device__ __forceinline__ void copy16_async(void* dst, const void* src) {
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
}

// First position of the ascending list[0 .. count) (entries < 0 lie behind the last) with an entry >= v;
// the whole warp searches, 32 probes a step.
__device__ __forceinline__ int first_at_least(const int32_t* list, int count, int v) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = count;  // the answer lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step + step - 1;
    bool ge = true;
    if (i < hi) {
      const int x = __ldg(list + i);
      ge = x >= v || x < 0;
    }
    const unsigned m = __ballot_sync(0xffffffffu, ge);
    if (m == 0) return hi;
    const int f = __ffs(m) - 1;
    hi = min(hi, lo + f * step + step - 1);
    lo = lo + f * step;
  }
  return lo;
}

// Slabs are `stride` bytes apart inside a page, their code rows row_bytes; a CTA moves 16 P bytes of a row of
// each slab of its group, and behind scales_at bytes of a slab its scale rows of sb bytes (0: none).
template <int P>
__global__ void __launch_bounds__(kCompactThreads) compact_rows_kernel(RowPages pages, int slabs, int group,
                                                                       int64_t stride, int row_bytes, int64_t page_bytes,
                                                                       int64_t scales_at, int sb,
                                                                       const int32_t* __restrict__ idx, int keep, int R,
                                                                       uint32_t* read_marks, uint32_t* turns) {
  constexpr int rb = 16 * P;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int first_wait, end_wait, late, turn;
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) turn = (int)atomicAdd(turns + (int64_t)blockIdx.z * gridDim.y + blockIdx.y, 1u);
    __syncthreads();
  }
  const int seg = gridDim.x > 1 ? turn : 0, t = blockIdx.z, s0 = blockIdx.y * group, ns = min(group, slabs - s0);
  const int j0 = seg * R, warp = threadIdx.x >> 5;
  const int32_t* list = idx + (int64_t)t * keep;
  uint32_t* marks = read_marks + ((int64_t)t * gridDim.y + blockIdx.y) * gridDim.x;
  uint8_t* const rows = smem;                                // [slab][row][rb]
  uint8_t* const sc = rows + (int64_t)ns * R * rb;           // [slab][row][sb]
  int4* const place = reinterpret_cast<int4*>(smem + (int64_t)group * R * (rb + sb));  // source page, slot; own page, slot
  bool any = false;
  for (int r = threadIdx.x; r < R; r += kCompactThreads) {
    const int j = j0 + r, src = j < keep ? __ldg(list + j) : -1;
    int64_t pf = -1, pt = -1;
    if (src >= 0 && src != j) {
      pf = kv4_page(pages, t, src, blockIdx.y == 0);
      pt = kv4_page(pages, t, j, false);
    }
    const bool ok = pf >= 0 && pt >= 0;
    any |= ok;
    place[r] = make_int4(ok ? (int)pf : -1, (int)((uint32_t)src % (uint32_t)pages.page_size), (int)pt,
                         (int)((uint32_t)j % (uint32_t)pages.page_size));
  }
  if (threadIdx.x == 0) late = 0;
  const bool moves = __syncthreads_or(any);
  uint8_t* const base = pages.base + s0 * stride;
  const int each = ns >= 8 ? 8 : 1;  // threads that share a row's scales
  if (moves) {
    for (int u = threadIdx.x; u < R * P; u += kCompactThreads) {
      const int r = u / P, piece = u % P;
      const int4 w = place[r];
      if (w.x < 0) continue;
      const uint8_t* p = base + w.x * page_bytes + (int64_t)w.y * row_bytes + piece * 16;
      for (int x = 0; x < ns; ++x) copy16_async(rows + ((int64_t)x * R + r) * rb + piece * 16, p + x * stride);
    }
    if (sb) {
      for (int u = threadIdx.x; u < R * each; u += kCompactThreads) {
        const int r = u / each;
        const int4 w = place[r];
        if (w.x < 0) continue;
        for (int x = u % each; x < ns; x += each) {
          const uint8_t* p = base + w.x * page_bytes + x * stride + scales_at + (int64_t)w.y * sb;
          const uint32_t q = (uint32_t)__cvta_generic_to_shared(sc + ((int64_t)x * R + r) * sb);
          if (sb == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(q), "l"(p) : "memory");
          else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(q), "l"(p) : "memory");
        }
      }
    }
    if (gridDim.x > 1 && warp < 2) {  // segments with sources in [j0, j0 + R), this one aside
      const int at = first_at_least(list, keep, warp ? j0 + R : j0);
      if ((threadIdx.x & 31) == 0) (warp ? end_wait : first_wait) = warp ? min(seg, (at + R - 1) / R) : at / R;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  __syncthreads();  // the segment has been read
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) {
      __threadfence();
      atomicExch(marks + seg, 1u);
    }
    if (!moves) return;
    if (warp == 0) {
      for (int x = first_wait + (int)threadIdx.x; x < end_wait; x += 32) {
        const volatile uint32_t* m = marks + x;
        if (*m) continue;
        uint64_t t0, t1;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        while (!*m) {
          __nanosleep(64);
          asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t1));
          if (t1 - t0 > kWaitLimitNs) {
            late = 1;
            break;
          }
        }
      }
      __threadfence();
    }
    __syncthreads();
    if (late) {
      if (threadIdx.x == 0) atomicExch(&g_compact_status, 1);
      return;
    }
  }
  for (int u = threadIdx.x; u < R * P; u += kCompactThreads) {
    const int r = u / P, piece = u % P;
    const int4 w = place[r];
    if (w.x < 0) continue;
    uint8_t* p = base + w.z * page_bytes + (int64_t)w.w * row_bytes + piece * 16;
#pragma unroll 4
    for (int x = 0; x < ns; ++x)
      *reinterpret_cast<uint4*>(p + x * stride) =
          *reinterpret_cast<const uint4*>(rows + ((int64_t)x * R + r) * rb + piece * 16);
  }
  if (sb) {
    for (int u = threadIdx.x; u < R * each; u += kCompactThreads) {
      const int r = u / each;
      const int4 w = place[r];
      if (w.x < 0) continue;
      for (int x = u % each; x < ns; x += each) {
        uint8_t* p = base + w.z * page_bytes + x * stride + scales_at + (int64_t)w.w * sb;
        const uint8_t* q = sc + ((int64_t)x * R + r) * sb;
        if (sb == 8) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(q);
        else *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(q);
      }
    }
  }
}

// How a compaction is cut up: rows of a segment, slabs of a group, segments, groups, shared memory.
struct CompactPlan {
  int R, group, segs, groups;
  size_t smem;
};

CompactPlan compact_plan(int T, int slabs, int rb, int sb, int keep) {
  CompactPlan p;
  const int row = rb + sb;
  int64_t room = kGroupBytes;
  // rows that fill the room, unless that leaves CTAs without any
  const int64_t fill = room / ((int64_t)slabs * row), share = (int64_t)T * keep / (4 * kGpuSms);
  p.R = (int)std::max<int64_t>(kSeg, std::min(std::min<int64_t>(fill, share) / 16 * 16, (int64_t)kOneSeg));
  if (keep <= kOneSeg && (int64_t)keep * row <= kOneSegBytes) {
    p.R = (keep + 15) / 16 * 16;
    room = std::max<int64_t>(room, (int64_t)p.R * row);
  }
  p.group = (int)std::min<int64_t>(slabs, std::max<int64_t>(1, room / ((int64_t)p.R * row)));
  // a call of few CTAs takes a slab each: their number is what its time depends on
  if ((int64_t)T * ((keep + p.R - 1) / p.R) * ((slabs + p.group - 1) / p.group) < kFewCtas) p.group = 1;
  p.segs = (keep + p.R - 1) / p.R;
  p.groups = (slabs + p.group - 1) / p.group;
  p.smem = (size_t)p.R * p.group * row + sizeof(int4) * p.R;
  return p;
}

// A mark for every segment, and behind them the segments handed out of every sequence and group.
size_t ws_words(int T, const CompactPlan& p) { return (size_t)T * p.groups * (p.segs + 1); }

}  // namespace

void launch_kv4_append(DType dt, const void* k, const void* v, int64_t ldk, int64_t ldv, const Kv4Pool& pool,
                       const int32_t* cu, const int32_t* start, int S, int rows, float kg, float vg, cudaStream_t s) {
  if (S <= 0 || rows <= 0) return;
  const unsigned grid = (unsigned)(((int64_t)rows * pool.Hkv * 2 * 4 + 255) / 256);
  auto run = [&](auto kernel) { kernel<<<grid, 256, 0, s>>>(k, v, ldk, ldv, pool, cu, start, S, rows, kg, vg); };
  if (pool.d == 128) dt == DType::BF16 ? run(kv4_append_kernel<128, DType::BF16>) : run(kv4_append_kernel<128, DType::F32>);
  else dt == DType::BF16 ? run(kv4_append_kernel<64, DType::BF16>) : run(kv4_append_kernel<64, DType::F32>);
}

void launch_kv4_read(DType dt, const Kv4Pool& pool, const int32_t* cu, const int32_t* start, int S, int rows,
                     float kg, float vg, void* k, void* v, cudaStream_t s) {
  if (S <= 0 || rows <= 0) return;
  const unsigned grid = (unsigned)(((int64_t)rows * pool.Hkv * 2 * 4 + 255) / 256);
  auto run = [&](auto kernel) { kernel<<<grid, 256, 0, s>>>(pool, cu, start, S, rows, kg, vg, k, v); };
  if (pool.d == 128) dt == DType::BF16 ? run(kv4_read_kernel<128, DType::BF16>) : run(kv4_read_kernel<128, DType::F32>);
  else dt == DType::BF16 ? run(kv4_read_kernel<64, DType::BF16>) : run(kv4_read_kernel<64, DType::F32>);
}

size_t compact_ws_bytes(int T, int keep, int slabs, int row, int sb) {
  const int rb = sb ? row : 64;
  slabs *= row / rb;
  const CompactPlan p = compact_plan(T, slabs, rb, sb, keep);
  return ws_words(T, p) * sizeof(uint32_t);
}

bool launch_compact_rows(const RowPages& pages, int slabs, int64_t slab_bytes, int row, int sb, const int32_t* idx,
                         int T, int keep, void* ws, cudaStream_t s) {
  if (T <= 0 || keep <= 0) return true;
  // a wide row without scales goes in columns of 64 bytes, as slabs of their own
  const int64_t page_bytes = slabs * slab_bytes, stride = sb ? slab_bytes : 64, scales_at = (int64_t)pages.page_size * row;
  const int rb = sb ? row : 64;
  slabs *= row / rb;
  const CompactPlan p = compact_plan(T, slabs, rb, sb, keep);
  uint32_t* const marks = static_cast<uint32_t*>(ws);
  uint32_t* const turns = marks + (size_t)T * p.groups * p.segs;
  if (p.segs > 1 && cudaMemsetAsync(ws, 0, sizeof(uint32_t) * ws_words(T, p), s) != cudaSuccess) return false;
  auto run = [&](auto kernel) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kOneSegBytes + 16384) != cudaSuccess)
      return false;
    constexpr int kMostZ = 65535;
    for (int t0 = 0; t0 < T; t0 += kMostZ) {
      RowPages q = pages;
      q.table += (int64_t)t0 * pages.max_pages;
      kernel<<<dim3(p.segs, p.groups, std::min(T - t0, kMostZ)), kCompactThreads, p.smem, s>>>(
          q, slabs, p.group, stride, row, page_bytes, scales_at, sb, idx + (int64_t)t0 * keep, keep, p.R,
          marks + (int64_t)t0 * p.groups * p.segs, turns + (int64_t)t0 * p.groups);
    }
    return true;
  };
  return rb == 32 ? run(compact_rows_kernel<2>) : run(compact_rows_kernel<4>);
}

int read_and_clear_compact_status() {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_compact_status, sizeof(int)) != cudaSuccess) return -1;
  if (v) {
    const int zero = 0;
    cudaMemcpyToSymbol(g_compact_status, &zero, sizeof(int));
  }
  return v;
}

MISA_BAD_ID_READER(read_and_clear_bad_ids_kv4_cache)

}  // namespace misa
