// Attention of single query tokens over a cache held in 4 bits (format in kv4.cuh):
//   s_{h,i} = scale k_scale (q_h . k_i),  out_h = v_scale sum_i softmax(s_h)_i v_i
// over the tokens i < n_t of query t's sequence, or over the tokens idx[t] of it (what the indexer
// selected); the H_q / H_kv query heads of a group share one key and value head.
//
// What bounds it: every code and scale of the attended rows is read once from HBM (1.125 d bytes a token
// and kv head, K and V), and each of them has to be widened and multiplied, so the instructions per byte
// are what can keep it from the memory's rate.  Both products run on mma.m16n8k16 with the tokens (then
// the head dimensions) as the 16 rows and the heads of a group as the 8 columns, so that the widened
// cache is the A operand and is never padded: 8 heads cost one product per 16 x 16 piece of the cache.
//   S^T [16 tokens x 8 heads] = K [16 x d] Q^T:   lane (r, c) widens its 16-byte chunk c of rows r, r+8
//   O^T [d x 8 heads] += V^T [d x 16] P^T:        lane (r, c) widens 8 bytes of tokens 2c, 2c+1, 2c+8, 2c+9,
//                                                  two tokens' nibbles merged into one byte beforehand
// e2m1 x e4m3 has 6 significant bits and lies in fp16's range, so the widened K and V are exact in fp16.
// The query row is scaled by a power of two into fp16's upper range, where a bf16 row is exact down to
// 2^-30 of its largest element; an fp32 row is split into two fp16 parts (22 bits), as are its weights.
// Softmax weights are rounded to fp16 (2^-12) for the product with V where the output is bf16; the sums,
// the maximum and the accumulators are fp32.
//
// Work: every warp streams its own tiles of 16 tokens through a ring of asynchronous copies and keeps
// its own running maximum, sum and output; the warps of a CTA join through shared memory, and the
// flattened (query, kv head, token) range is cut into equal pieces, one per CTA, whose partial results a
// second kernel joins where a piece ends inside a head's tokens.
#include <algorithm>

#include "kernels.cuh"
#include "kv4.cuh"
#include "tmap.cuh"

namespace misa {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;              // tokens of a warp's step
constexpr int kUnit = kWarps * kTile;  // tokens of a CTA's step: the grain of the split
constexpr int kMaxT = 1024;            // queries per launch
constexpr int kStages = 4;
constexpr int kMaxCtas = 1024;         // bound on the grid, for workspace sizes that ask no device
// Weights are kept scaled by 2^kLift against the running maximum, which may lag the true one by
// 2^kSlack: 2^15 at most, and what fp16 loses at the bottom lies below 2^-35 of the largest weight.
constexpr float kLift = 11.f, kSlack = 4.f;

template <int D>
struct Stage {
  static constexpr int kCodes = kTile * D / 2;    // bytes of one side's codes
  static constexpr int kScales = kTile * D / 16;  // bytes of one side's scales
  static constexpr int kV = kCodes, kKs = 2 * kCodes, kVs = kKs + kScales, kMask = kVs + kScales;
  static constexpr int kBytes = kMask + 16;
};

struct AttnArgs {
  const void* q;
  Kv4Pool pool;
  const int32_t* n;
  const int32_t* idx;  // [T][P] or null
  int T, L, P, Hq, G, groups;  // groups: blocks of 8 NT heads per kv head
  float scale, v_scale;        // scale carries log2(e) and k_scale
  void* out;
  float* lse;       // [T][Hq] natural log, or null
  float* lse2;      // [T][Hq] base 2 (weights wanted), or null
  float* logits;    // [T][Hq][ldS] base 2, or null
  int64_t ldS;
  float* part;      // partial results: [slot][8 NT][D] sums, then [slot][8 NT][2] maximum and sum
  float* part_ml;
  uint64_t* pre;    // [T + 1] first unit of each query
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t low2(uint32_t x) { return __byte_perm(x, x, 0x1010); }
__device__ __forceinline__ uint32_t high2(uint32_t x) { return __byte_perm(x, x, 0x3232); }

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack_half2(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// Copies the first n of BYTES bytes and fills the rest with zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int n) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Units (of kUnit positions) of every query and their running sum: pre[0 .. T].
__device__ __forceinline__ void unit_prefix(const AttnArgs& a, uint64_t* pre, uint64_t* tot) {
  const int per = (a.T + kThreads - 1) / kThreads;
  const int b0 = min(a.T, (int)threadIdx.x * per), b1 = min(a.T, b0 + per);
  uint64_t local = 0;
  for (int t = b0; t < b1; ++t) {
    const int nt = clamp_len(__ldg(a.n + t), a.L);
    const int len = a.idx ? (nt > 0 ? a.P : 0) : nt;
    local += (uint64_t)((len + kUnit - 1) / kUnit) * (a.pool.Hkv * a.groups);
    pre[t + 1] = local;
  }
  tot[threadIdx.x] = local;
  __syncthreads();
  uint64_t before = 0;
  for (int i = 0; i < (int)threadIdx.x; ++i) before += tot[i];
  for (int t = b0; t < b1; ++t) pre[t + 1] += before;
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
}

template <int D, int NT, int SPLIT, bool GATHER>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 2) kv4_attn_kernel(const AttnArgs a) {
  using St = Stage<D>;
  constexpr int KS = D / 16;      // k-steps of S, and 16-row pieces of O
  constexpr int RB = D / 2;       // bytes of a code row
  constexpr int HB = 8 * NT;      // heads of an item
  constexpr int kRing = kWarps * kStages * St::kBytes;
  constexpr int kJoin = kWarps * HB * (D + 2) * 4;
  __shared__ __align__(16) uint8_t ring[kRing > kJoin ? kRing : kJoin];
  __shared__ uint64_t pre[kMaxT + 1];
  __shared__ uint64_t tot[kThreads];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  unit_prefix(a, pre, tot);
  if (blockIdx.x == 0)
    for (int t = threadIdx.x; t <= a.T; t += kThreads) a.pre[t] = pre[t];
  const uint64_t W = pre[a.T];
  const uint64_t grid = W < gridDim.x ? W : gridDim.x;
  if (blockIdx.x >= grid) return;
  uint64_t pos = W * blockIdx.x / grid;
  const uint64_t end = W * (blockIdx.x + 1) / grid;
  const int items = a.pool.Hkv * a.groups;
  const uint32_t my_ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + warp * kStages * St::kBytes;
  uint8_t* const my_ptr = ring + warp * kStages * St::kBytes;
  int t = 0;
  {
    int hi = a.T - 1;  // last query with pre[t] <= pos
    while (t < hi) {
      const int mid = (t + hi + 1) >> 1;
      if (pre[mid] <= pos) t = mid;
      else hi = mid - 1;
    }
  }
  while (pos < end) {
    while (pre[t + 1] <= pos) ++t;
    const uint32_t units = (uint32_t)((pre[t + 1] - pre[t]) / items);  // of one item
    const uint64_t at = pos - pre[t];
    const int item = (int)(at / units);
    const uint32_t u0 = (uint32_t)(at - (uint64_t)item * units);
    const uint32_t u1 = (uint32_t)min((uint64_t)units, u0 + (end - pos));
    pos += u1 - u0;
    const int hk = item / a.groups, hg = item - hk * a.groups;
    const int nt = clamp_len(__ldg(a.n + t), a.L);
    const int len = GATHER ? a.P : nt;
    const int heads = min(HB, a.G - hg * HB);           // of this item
    const int64_t h0 = (int64_t)t * a.Hq + hk * a.G + hg * HB;

    // query fragments: step j, lane (r, c): elements 16 j + 4 c .. + 3 of head r (+ 8)
    uint32_t qf[SPLIT][NT][KS][2];
    float mul[NT][2];  // logits of heads 2c, 2c + 1 per unit of the product
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      float f[KS][4];
      float top = 0.f;
      const int head = x * 8 + r;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const int64_t e = (h0 + head) * D + 16 * j + 4 * c;
        if (head >= heads) {
          f[j][0] = f[j][1] = f[j][2] = f[j][3] = 0.f;
        } else if (SPLIT == 1) {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) + e));
          f[j][0] = bf16_lo(u.x);
          f[j][1] = bf16_hi(u.x);
          f[j][2] = bf16_lo(u.y);
          f[j][3] = bf16_hi(u.y);
        } else {
          const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + e));
          f[j][0] = u.x;
          f[j][1] = u.y;
          f[j][2] = u.z;
          f[j][3] = u.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(f[j][i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^up brings the largest element into [2^13, 2^14)
      const int ex = (int)((__float_as_uint(top) >> 23) & 255u) - 127;
      const int up = top == 0.f || ex == 128 ? 0 : min(126, 13 - ex);
      const float by = __uint_as_float((uint32_t)(up + 127) << 23);
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float y0 = f[j][2 * i] * by, y1 = f[j][2 * i + 1] * by;
          qf[0][x][j][i] = pack_half2(y0, y1);
          if (SPLIT == 2) {
            const float2 b = unpack_half2(qf[0][x][j][i]);
            qf[SPLIT - 1][x][j][i] = pack_half2(y0 - b.x, y1 - b.y);
          }
        }
      const float down = a.scale * __uint_as_float((uint32_t)(127 - up) << 23);  // of head r
      mul[x][0] = __shfl_sync(0xffffffffu, down, 8 * c);
      mul[x][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
    }

    float o[NT][KS][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      m[x][0] = m[x][1] = -INFINITY;
      l[x][0] = l[x][1] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i) o[x][i][0] = o[x][i][1] = o[x][i][2] = o[x][i][3] = 0.f;
    }

    // warp w takes tiles w, w + kWarps, ... of the segment
    const int p0 = (int)u0 * kUnit, tiles = (int)(u1 - u0);
    const int64_t slab = (int64_t)(2 * hk) * a.pool.slab_bytes();
    // row lookups run ahead of the copies: the token of tile i + 2 and the page of tile i + 1
    int tok_next = -1, tok_now = -1;
    int64_t pg_now = -1;
    auto token_of = [&](int i) -> int {
      if (i >= tiles) return -1;
      const int p = p0 + (i * kWarps + warp) * kTile + (GATHER ? (lane & 15) : 0);
      if (p >= len) return -1;
      if (!GATHER) return p;
      const int s = __ldg(a.idx + (int64_t)t * a.P + p);
      count_bad_id(kBadCandidate, s != -1 && (s < 0 || s >= nt) && lane < 16 && item == 0);
      return s >= 0 && s < nt ? s : -1;
    };
    auto page_of = [&](int tok) -> int64_t {
      return kv4_page(a.pool, t, tok, item == 0 && (GATHER ? lane < 16 : lane == 0));
    };
    // copies tile i into stage st; tok and pg are its first token (gathered: of row lane & 15) and page
    auto issue = [&](int i, int st, int tok, int64_t pg) {
      if (i < tiles) {
        const uint32_t dst = my_ring + st * St::kBytes;
        const int sl = tok < 0 ? 0 : (int)((uint32_t)tok % (uint32_t)a.pool.page_size);
        if (!GATHER) {
          const int rows = pg < 0 ? 0 : min(kTile, len - tok);
          const uint8_t* base = a.pool.base + (pg < 0 ? 0 : pg * a.pool.page_bytes()) + slab;
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const uint8_t* src = base + side * a.pool.slab_bytes() + (int64_t)sl * RB;
#pragma unroll
            for (int y = lane; y < St::kCodes / 16; y += 32)
              copy_async<16>(dst + side * St::kV + y * 16, src + y * 16, y * 16 / RB < rows ? 16 : 0);
          }
          constexpr int SC = St::kScales / 16;  // 16-byte pieces of one side's scales
          if (lane < 2 * SC) {
            const int side = lane / SC, y = lane % SC;
            copy_async<16>(dst + St::kKs + side * St::kScales + y * 16,
                           base + side * a.pool.slab_bytes() + a.pool.scales_at() + (int64_t)sl * KS + y * 16,
                           max(0, min(16, rows * KS - y * 16)));  // rows past the prefix: zero scales
          }
          if (lane == 0)
            *reinterpret_cast<uint32_t*>(my_ptr + st * St::kBytes + St::kMask) = (1u << rows) - 1u;
        } else {
          const bool there = pg >= 0;
          const uint32_t mask = __ballot_sync(0xffffffffu, there) & 0xffffu;
          const int64_t row = there ? pg * a.pool.page_bytes() + slab : 0;
          constexpr int CR = RB / 16;  // 16-byte pieces of a code row
#pragma unroll
          for (int y = 0; y < kTile * CR / 32; ++y) {
            const int at_row = (y * 32 + lane) / CR, piece = (y * 32 + lane) % CR;
            const int64_t b = __shfl_sync(0xffffffffu, row, at_row);
            const int s1 = __shfl_sync(0xffffffffu, sl, at_row);
            const uint8_t* src = a.pool.base + b + (int64_t)s1 * RB + piece * 16;
            const bool ok = (mask >> at_row) & 1u;
            copy_async<16>(dst + at_row * RB + piece * 16, src, ok ? 16 : 0);
            copy_async<16>(dst + St::kV + at_row * RB + piece * 16, ok ? src + a.pool.slab_bytes() : src, ok ? 16 : 0);
          }
          const int side = lane >> 4;
          copy_async<KS>(dst + St::kKs + side * St::kScales + (lane & 15) * KS,
                         a.pool.base + row + side * a.pool.slab_bytes() + a.pool.scales_at() + (int64_t)sl * KS,
                         there ? KS : 0);
          if (lane == 0) *reinterpret_cast<uint32_t*>(my_ptr + st * St::kBytes + St::kMask) = mask;
        }
      }
      copy_commit();
    };
    tok_now = token_of(0);
    tok_next = token_of(1);
    pg_now = page_of(tok_now);
    auto advance = [&](int i, int st) {  // issues tile i; its token and page are in the *_now values
      issue(i, st, tok_now, pg_now);
      tok_now = tok_next;
      pg_now = page_of(tok_now);
      tok_next = token_of(i + 2);
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) advance(i, i);

#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      const int st = i % kStages;
      copy_wait<kStages - 2>();
      __syncwarp();
      advance(i + kStages - 1, (i + kStages - 1) % kStages);
      const uint8_t* sp = my_ptr + st * St::kBytes;
      const uint32_t mask = *reinterpret_cast<const uint32_t*>(sp + St::kMask);

      // S^T = K Q^T
      float s[NT][4];
#pragma unroll
      for (int x = 0; x < NT; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
      uint32_t ka[KS / 2], kb[KS / 2], sa[KS / 4], sb[KS / 4];
      if constexpr (D == 128) {
        const uint4 u = *reinterpret_cast<const uint4*>(sp + r * RB + c * 16);
        const uint4 v = *reinterpret_cast<const uint4*>(sp + (r + 8) * RB + c * 16);
        ka[0] = u.x, ka[1] = u.y, ka[2] = u.z, ka[3] = u.w;
        kb[0] = v.x, kb[1] = v.y, kb[2] = v.z, kb[3] = v.w;
        const uint2 e = *reinterpret_cast<const uint2*>(sp + St::kKs + r * KS);
        const uint2 f = *reinterpret_cast<const uint2*>(sp + St::kKs + (r + 8) * KS);
        sa[0] = e.x, sa[1] = e.y, sb[0] = f.x, sb[1] = f.y;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(sp + r * RB + c * 8);
        const uint2 v = *reinterpret_cast<const uint2*>(sp + (r + 8) * RB + c * 8);
        ka[0] = u.x, ka[1] = u.y;
        kb[0] = v.x, kb[1] = v.y;
        sa[0] = *reinterpret_cast<const uint32_t*>(sp + St::kKs + r * KS);
        sb[0] = *reinterpret_cast<const uint32_t*>(sp + St::kKs + (r + 8) * KS);
      }
#pragma unroll
      for (int w = 0; w < KS / 2; ++w) {
        uint32_t x0[4], x1[4];
        e2m1x8_to_half2(ka[w], x0[0], x0[1], x0[2], x0[3]);
        e2m1x8_to_half2(kb[w], x1[0], x1[1], x1[2], x1[3]);
        const uint32_t e = e4m3x2_to_half2((uint16_t)(sa[w / 2] >> (16 * (w & 1))));
        const uint32_t f = e4m3x2_to_half2((uint16_t)(sb[w / 2] >> (16 * (w & 1))));
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t ee = y ? high2(e) : low2(e), ff = y ? high2(f) : low2(f);
          const uint32_t a0 = hmul2(x0[2 * y], ee), a1 = hmul2(x1[2 * y], ff), a2 = hmul2(x0[2 * y + 1], ee),
                         a3 = hmul2(x1[2 * y + 1], ff);
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int z = 0; z < SPLIT; ++z)
              mma_f16(s[x], a0, a1, a2, a3, qf[z][x][2 * w + y][0], qf[z][x][2 * w + y][1]);
        }
      }
      // logits in base 2, rows without a token minus infinity; s[x][0..1] row r, s[x][2..3] row r + 8
      const bool v0 = (mask >> r) & 1u, v1 = (mask >> (r + 8)) & 1u;
      bool raise = false;
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        s[x][0] = v0 ? s[x][0] * mul[x][0] : -INFINITY;
        s[x][1] = v0 ? s[x][1] * mul[x][1] : -INFINITY;
        s[x][2] = v1 ? s[x][2] * mul[x][0] : -INFINITY;
        s[x][3] = v1 ? s[x][3] * mul[x][1] : -INFINITY;
        raise |= fmaxf(s[x][0], s[x][2]) > m[x][0] + kSlack || fmaxf(s[x][1], s[x][3]) > m[x][1] + kSlack;
      }
      if (a.logits) {
        const int p = p0 + (i * kWarps + warp) * kTile + r;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int head = x * 8 + 2 * c + y;
            if (head < heads) {
              float* row = a.logits + (h0 + head) * a.ldS + p;
              row[0] = s[x][y];
              row[8] = s[x][2 + y];
            }
          }
      }
      // the running maximum is raised only when a logit passes it by kSlack
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float top = fmaxf(s[x][y], s[x][2 + y]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float next = fmaxf(m[x][y], top);
            const float f = m[x][y] == next ? 1.f : exp2_fast(m[x][y] - next);
            m[x][y] = next;
            l[x][y] *= f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[x][k][y] *= f;
              o[x][k][2 + y] *= f;
            }
          }
      }
      uint32_t pb[SPLIT][NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const float z0 = m[x][0] == -INFINITY ? 0.f : m[x][0] - kLift, z1 = m[x][1] == -INFINITY ? 0.f : m[x][1] - kLift;
        const float w0 = exp2_fast(s[x][0] - z0), w1 = exp2_fast(s[x][1] - z1);
        const float w2 = exp2_fast(s[x][2] - z0), w3 = exp2_fast(s[x][3] - z1);
        l[x][0] += w0 + w2;
        l[x][1] += w1 + w3;
        const uint32_t h0_ = pack_half2(w0, w1), h1_ = pack_half2(w2, w3);
        pb[0][x][0] = transpose8(h0_);
        pb[0][x][1] = transpose8(h1_);
        if (SPLIT == 2) {
          const float2 b0 = unpack_half2(h0_), b1 = unpack_half2(h1_);
          pb[SPLIT - 1][x][0] = transpose8(pack_half2(w0 - b0.x, w1 - b0.y));
          pb[SPLIT - 1][x][1] = transpose8(pack_half2(w2 - b1.x, w3 - b1.y));
        }
      }

      // O^T += V^T P^T: byte i of a lane's chunk holds piece i's rows r (low nibble) and r + 8 (high)
      const uint8_t* vp = sp + St::kV + r * (RB / 8);
      const uint8_t* vs = sp + St::kVs + (r & 1) * (KS / 2);
#pragma unroll
      for (int w = 0; w < KS / 4; ++w) {  // 4 pieces, 2 blocks of 16 elements
        uint32_t lo[2][4], hi[2][4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {  // tokens 2c, 2c + 1, then 8 further
          const int ta = 2 * c + 8 * hf;
          const uint32_t xa = *reinterpret_cast<const uint32_t*>(vp + ta * RB + 4 * w);
          const uint32_t xb = *reinterpret_cast<const uint32_t*>(vp + (ta + 1) * RB + 4 * w);
          e2m1x8_to_half2((xa & 0x0f0f0f0fu) | ((xb << 4) & 0xf0f0f0f0u), lo[hf][0], lo[hf][1], lo[hf][2], lo[hf][3]);
          e2m1x8_to_half2(((xa >> 4) & 0x0f0f0f0fu) | (xb & 0xf0f0f0f0u), hi[hf][0], hi[hf][1], hi[hf][2], hi[hf][3]);
          const uint32_t ea = *reinterpret_cast<const uint16_t*>(vs + ta * KS + 2 * w);
          const uint32_t eb = *reinterpret_cast<const uint16_t*>(vs + (ta + 1) * KS + 2 * w);
          const uint32_t ab = __byte_perm(ea, eb, 0x5140);  // scales of block 0: a, b; of block 1: a, b
          const uint32_t f0 = e4m3x2_to_half2((uint16_t)ab), f1 = e4m3x2_to_half2((uint16_t)(ab >> 16));
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            lo[hf][y] = hmul2(lo[hf][y], y < 2 ? f0 : f1);
            hi[hf][y] = hmul2(hi[hf][y], y < 2 ? f0 : f1);
          }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int z = 0; z < SPLIT; ++z)
              mma_f16(o[x][4 * w + y], lo[0][y], hi[0][y], lo[1][y], hi[1][y], pb[z][x][0], pb[z][x][1]);
      }
    }
    copy_wait<0>();
    __syncthreads();  // the ring becomes the join's scratch

    // join the warps: sums [warp][head][D], then maximum and sum
    float* sums = reinterpret_cast<float*>(ring);
    float* ml = sums + kWarps * HB * D;
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float v = l[x][y];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        const int head = x * 8 + 2 * c + y;
        float* dst = sums + (warp * HB + head) * D;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int dim = 16 * ((KS / 2) * (r & 1) + k / 2) + 4 * (r >> 1) + 2 * (k & 1);
          *reinterpret_cast<float2*>(dst + dim) = make_float2(o[x][k][y], o[x][k][2 + y]);
        }
        if (r == 0) {
          ml[(warp * HB + head) * 2] = m[x][y];
          ml[(warp * HB + head) * 2 + 1] = v;
        }
      }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == units;
    const int64_t slot = (int64_t)blockIdx.x + (int64_t)t * items + item;
    for (int e = threadIdx.x; e < heads * (D / 4); e += kThreads) {
      const int head = e / (D / 4), d4 = e % (D / 4) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[(w * HB + head) * 2]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = ml[(w * HB + head) * 2];
        if (ml[(w * HB + head) * 2 + 1] == 0.f) continue;  // a warp that saw no token
        const float f = exp2_fast(mw - top);
        sum += f * ml[(w * HB + head) * 2 + 1];
        const float4 v = *reinterpret_cast<const float4*>(sums + (w * HB + head) * D + d4);
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
      }
      if (whole) {
        const float inv = sum == 0.f ? 0.f : a.v_scale / sum;
        const int64_t at_out = (h0 + head) * D + d4;
        if (SPLIT == 1) {
          __nv_bfloat162* p = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + at_out);
          p[0] = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
          p[1] = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        } else {
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at_out) =
              make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        }
        if (d4 == 0) {
          const float z = sum == 0.f ? -INFINITY : top + log2f(sum) - kLift;
          if (a.lse) a.lse[h0 + head] = z * 0.693147180559945309f;
          if (a.lse2) a.lse2[h0 + head] = z;
        }
      } else {
        *reinterpret_cast<float4*>(a.part + (slot * HB + head) * D + d4) = acc;
        if (d4 == 0) {
          a.part_ml[(slot * HB + head) * 2] = top;
          a.part_ml[(slot * HB + head) * 2 + 1] = sum;
        }
      }
    }
    __syncthreads();  // before the next segment's copies overwrite the scratch
  }
}

// Joins the pieces of every (query, head) whose tokens more than one CTA took; also writes the heads
// of queries that attend to nothing.  One warp per head.
template <int D, int SPLIT>
__global__ void __launch_bounds__(256) kv4_join_kernel(const AttnArgs a, int HB, int64_t ctas) {
  pdl_wait();
  const int64_t hd = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (hd >= (int64_t)a.T * a.Hq) return;
  const int t = (int)(hd / a.Hq), hq = (int)(hd % a.Hq);
  const int hk = hq / a.G, hr = hq % a.G, head = hr % HB;
  const int items = a.pool.Hkv * a.groups, item = hk * a.groups + hr / HB;
  const uint64_t W = a.pre[a.T], first = a.pre[t];
  const uint64_t units = (a.pre[t + 1] - first) / items;
  constexpr int E = D / 32;  // output elements of a lane
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float top = -INFINITY, sum = 0.f;
  if (units > 0) {
    const uint64_t grid = W < (uint64_t)ctas ? W : (uint64_t)ctas;
    const uint64_t p0 = first + item * units, p1 = p0 + units;
    const int64_t c0 = (int64_t)(((p0 + 1) * grid - 1) / W), c1 = (int64_t)((p1 * grid - 1) / W);
    if (c0 == c1) return;  // one CTA had the whole head
    const int64_t slot0 = c0 + (int64_t)t * items + item;
    const int pieces = (int)(c1 - c0 + 1);
    for (int i = lane; i < pieces; i += 32) top = fmaxf(top, a.part_ml[((slot0 + i) * HB + head) * 2]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 4
    for (int i = 0; i < pieces; ++i) {
      const int64_t at = (slot0 + i) * HB + head;
      const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
      const float* p = a.part + at * D + lane * E;
      const float f = ml.y == 0.f ? 0.f : exp2_fast(ml.x - top);
      sum += f * ml.y;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += f * p[e];
    }
  }
  const float inv = sum == 0.f ? 0.f : a.v_scale / sum;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (SPLIT == 1) static_cast<__nv_bfloat16*>(a.out)[hd * D + lane * E + e] = __float2bfloat16_rn(acc[e] * inv);
    else static_cast<float*>(a.out)[hd * D + lane * E + e] = acc[e] * inv;
  }
  if (lane == 0) {
    const float z = sum == 0.f ? -INFINITY : top + log2f(sum) - kLift;
    if (a.lse) a.lse[hd] = z * 0.693147180559945309f;
    if (a.lse2) a.lse2[hd] = z;
  }
}

// acc[t, i] += sum over the heads of token i's weight, from the logits and every head's log-sum.
// Selected tokens are added atomically: a token that a list names twice gets both of its (equal)
// weights, in either order the same sum.
__global__ void __launch_bounds__(256) kv4_weights_kernel(const AttnArgs a, float* __restrict__ acc, int64_t ld) {
  pdl_wait();
  const int t = blockIdx.y;
  const int p = blockIdx.x * 256 + threadIdx.x;
  const int nt = clamp_len(a.n[t], a.L);
  const int len = a.idx ? a.P : nt;
  if (p >= len) return;
  const int s = a.idx ? a.idx[(int64_t)t * a.P + p] : p;
  if (s < 0 || s >= nt) return;
  const float* row = a.logits + (int64_t)t * a.Hq * a.ldS + p;
  const float* z = a.lse2 + (int64_t)t * a.Hq;
  float w = 0.f;
#pragma unroll 8
  for (int h = 0; h < a.Hq; ++h) {
    const float lz = z[h], x = row[h * a.ldS];
    w += lz == -INFINITY ? 0.f : exp2_fast(x - lz);
  }
  float* dst = acc + (int64_t)t * ld + s;
  if (a.idx) atomicAdd(dst, w);
  else *dst += w;
}

int heads_per_item(int G) { return G > 8 ? 16 : 8; }

int64_t attn_ctas(int T, int P, int Hkv, int G) {
  const int HB = heads_per_item(G);
  const int64_t most = (int64_t)T * Hkv * ((G + HB - 1) / HB) * ((P + kUnit - 1) / kUnit);
  const int64_t full = std::min<int64_t>((int64_t)sm_count() * (HB == 8 ? 4 : 2), kMaxCtas);
  return std::min(most, full);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <int D, int NT, int SPLIT>
void launch_attn(const AttnArgs& a, float* acc, int64_t ld_acc, int64_t ctas, cudaStream_t s) {
  if (ctas > 0) {
    if (a.idx) kv4_attn_kernel<D, NT, SPLIT, true><<<(unsigned)ctas, kThreads, 0, s>>>(a);
    else kv4_attn_kernel<D, NT, SPLIT, false><<<(unsigned)ctas, kThreads, 0, s>>>(a);
  }
  const int64_t hd = (int64_t)a.T * a.Hq;
  launch_pdl(kv4_join_kernel<D, SPLIT>, dim3((unsigned)((hd + 7) / 8)), dim3(256), 0, s, a, 8 * NT, ctas);
  if (acc) launch_pdl(kv4_weights_kernel, dim3((a.P + 255) / 256, a.T), dim3(256), 0, s, a, acc, ld_acc);
}

}  // namespace

size_t kv4_attention_ws_bytes(int T, int P, int Hq, int Hkv, int d, bool weights) {
  const int G = Hq / Hkv, HB = heads_per_item(G);
  const int Tc = T < kMaxT ? T : kMaxT;
  const int64_t slots = kMaxCtas + (int64_t)Tc * Hkv * ((G + HB - 1) / HB);
  size_t b = up256(sizeof(uint64_t) * (kMaxT + 1)) + up256(sizeof(float) * slots * HB * d) + up256(sizeof(float) * slots * HB * 2);
  if (weights) b += up256(sizeof(float) * (size_t)Tc * Hq) + up256(sizeof(float) * (size_t)Tc * Hq * ((P + 63) / 64 * 64));
  return b;
}

void launch_kv4_attention(DType dt, const void* q, const Kv4Pool& pool, const int32_t* n, const int32_t* idx, int T,
                          int L, int P, int Hq, float scale, float k_scale, float v_scale, void* out, float* lse,
                          float* acc, int64_t ld_acc, void* ws, cudaStream_t s) {
  const int G = Hq / pool.Hkv, HB = heads_per_item(G);
  const size_t elt = dt == DType::BF16 ? 2 : 4;
  for (int t0 = 0; t0 < T; t0 += kMaxT) {
    const int Tc = T - t0 < kMaxT ? T - t0 : kMaxT;
    AttnArgs a;
    a.q = static_cast<const char*>(q) + elt * t0 * (size_t)Hq * pool.d;
    a.pool = pool;
    a.pool.table = pool.table + (int64_t)t0 * pool.max_pages;
    a.n = n + t0;
    a.idx = idx ? idx + (int64_t)t0 * P : nullptr;
    a.T = Tc;
    a.L = L;
    a.P = idx ? P : L;
    a.Hq = Hq;
    a.G = G;
    a.groups = (G + HB - 1) / HB;
    a.scale = scale * k_scale * 1.44269504088896341f;
    a.v_scale = v_scale;
    a.out = static_cast<char*>(out) + elt * t0 * (size_t)Hq * pool.d;
    a.lse = lse ? lse + (int64_t)t0 * Hq : nullptr;
    const int64_t ctas = attn_ctas(Tc, a.P, pool.Hkv, G);
    const int64_t slots = kMaxCtas + (int64_t)Tc * pool.Hkv * a.groups;
    char* p = static_cast<char*>(ws);
    a.pre = reinterpret_cast<uint64_t*>(p);
    p += up256(sizeof(uint64_t) * (kMaxT + 1));
    a.part = reinterpret_cast<float*>(p);
    p += up256(sizeof(float) * slots * HB * pool.d);
    a.part_ml = reinterpret_cast<float*>(p);
    p += up256(sizeof(float) * slots * HB * 2);
    a.lse2 = nullptr;
    a.logits = nullptr;
    a.ldS = 0;
    float* ac = nullptr;
    if (acc) {
      a.lse2 = reinterpret_cast<float*>(p);
      p += up256(sizeof(float) * (size_t)Tc * Hq);
      a.logits = reinterpret_cast<float*>(p);
      a.ldS = (a.P + 63) / 64 * 64;
      ac = acc + (int64_t)t0 * ld_acc;
    }
    const bool f32 = dt == DType::F32;
    if (pool.d == 128) {
      if (HB == 8) f32 ? launch_attn<128, 1, 2>(a, ac, ld_acc, ctas, s) : launch_attn<128, 1, 1>(a, ac, ld_acc, ctas, s);
      else f32 ? launch_attn<128, 2, 2>(a, ac, ld_acc, ctas, s) : launch_attn<128, 2, 1>(a, ac, ld_acc, ctas, s);
    } else {
      if (HB == 8) f32 ? launch_attn<64, 1, 2>(a, ac, ld_acc, ctas, s) : launch_attn<64, 1, 1>(a, ac, ld_acc, ctas, s);
      else f32 ? launch_attn<64, 2, 2>(a, ac, ld_acc, ctas, s) : launch_attn<64, 2, 1>(a, ac, ld_acc, ctas, s);
    }
  }
}

MISA_BAD_ID_READER(read_and_clear_bad_ids_kv4_attn)

}  // namespace misa
