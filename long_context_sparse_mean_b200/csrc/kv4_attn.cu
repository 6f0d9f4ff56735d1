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
// K enters its product as bare codes, one block of 16 elements a step, and the block's scale multiplies
// the result in fp32 (both rows of a lane: 4 multiply-adds a step, on twice as many lanes as the 4 fp16
// multiplications of the operand would have); V's scales run along the contraction and go onto the codes:
// e2m1 x e4m3 has 6 significant bits and lies in fp16's range, so both operands are exact.
// The query row is scaled by a power of two into fp16's upper range, where a bf16 row is exact down to
// 2^-30 of its largest element; an fp32 row is split into two fp16 parts (22 bits), as are its weights.
// Softmax weights are rounded to fp16 (half a step: 2^-11 of the weight) for the product with V where the output
// is bf16; the sums, the maximum and the accumulators are fp32.
//
// Work: every warp streams its own steps of 32 tokens through two buffers of asynchronous copies and keeps its
// own running maximum, sum and output; the warps of a CTA join through shared memory, and the flattened (query,
// kv head, token) range is cut into equal pieces, one per CTA, whose partial results a second kernel joins
// where a piece ends inside a head's tokens.  Weights to be summed need the finished log-sums: the logits are
// kept, and a third kernel turns them into weights.
//
// Measured: 16 queries of 64 heads over 120K to 128K tokens on 8 kv heads of d = 128 take 463 us by themselves, 5.0
// TB/s of cache (0.77 of the measured copy rate), 526 us in a long run of calls on changing inputs; 0.64
// instructions a clock and scheduler: of 467 us, 393 without the copies, 465 without the widening of K, 428 of V,
// 469 without the products.  Slower: five CTAs an SM at 96 registers 495, K and V refilled by themselves 494, bulk
// copies of 128 bytes to 1 KB 561, of whole pages shared by two warps 526.  32 queries of 32 heads over up to 16K tokens: 41 us, joins 8 and weights 10 us; 2048 selected
// tokens of 32 queries (64 heads): 54 us with its joins for 75 MB in rows of 64 and 8 bytes from anywhere, 64 with the weights.
#include <algorithm>

#include "kernels.cuh"
#include "kv4.cuh"
#include "tmap.cuh"

namespace misa {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSub = 16;               // tokens of a product's 16 rows; pages hold whole pieces of 16
constexpr int kTile = 2 * kSub;        // tokens of a warp's step
constexpr int kUnit = kWarps * kTile;  // tokens of a CTA's step: the grain of the split
// Units that an item's start and end take as long as, for the even split: without them the CTAs that go from one
// item to the next end last (64 queries of up to 16K tokens: 112 us, with one 104, two 102, four 104).  Units of
// selected tokens take longer, and each CTA few of them; which is better depends on the batch (2048 tokens of 64
// heads on 8: 32 queries 53.6 us without, 55.8 with two, 16 queries 34.8 and 32.9, 8 queries 24.7 and 22.6; 1000 of
// 32 heads on 4, 100 queries: 47.4 and 48.5), and large batches decided it.
__host__ __device__ constexpr uint32_t item_cost(bool selected) { return selected ? 0u : 2u; }
constexpr int kMaxT = 256;             // queries per launch,
// fewer where their logits, kept to sum weights, would take more than this (those of 256 queries of 64 heads over
// 128K tokens take 8 GiB, which a workspace then keeps)
constexpr size_t kLogitBytes = (size_t)1 << 30;
constexpr int kMaxCtas = 1024;         // bound on the grid, for workspace sizes that ask no device
// Weights are kept scaled by 2^kLift against the running maximum, which may lag the true one by
// 2^kSlack: 2^15 at most, and what fp16 loses at the bottom lies below 2^-35 of the largest weight.
constexpr float kLift = 11.f, kSlack = 4.f;
// A warp's buffer for one step: two pieces of 16 tokens, each [K codes][V codes][K scales][V scales].
template <int D>
struct Stage {
  static constexpr int kCodes = kSub * D / 2;    // bytes of one side's codes
  static constexpr int kScales = kSub * D / 16;  // bytes of one side's scales
  static constexpr int kV = kCodes, kKs = 2 * kCodes, kVs = kKs + kScales, kPiece = kVs + kScales;
  static constexpr int kBytes = 2 * kPiece;
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
  uint32_t page_mul;  // ceil(2^32 / (page_size / 16)), 0 for pages of 16: logical pages without a division
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

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack_half2(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte i of four e4m3 numbers (not negative) as fp32, times 2^-120.
__device__ __forceinline__ float scale_bits(uint32_t x, int i) {
  return __uint_as_float((i < 3 ? x << (20 - 8 * i) : x >> 4) & 0x07f00000u);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Units (of kUnit positions) of every query, item_cost more for every item, and their running sum: pre[0 .. T].
template <bool GATHER>
__device__ __forceinline__ void unit_prefix(const AttnArgs& a, uint64_t* pre, uint64_t* tot) {
  const int per = (a.T + kThreads - 1) / kThreads;
  const int b0 = min(a.T, (int)threadIdx.x * per), b1 = min(a.T, b0 + per);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t local = 0;
  for (int t = b0; t < b1; ++t) {
    const int nt = clamp_len(__ldg(a.n + t), a.L);
    const int len = a.idx ? (nt > 0 ? a.P : 0) : nt;
    if (len > 0) local += (uint64_t)((len + kUnit - 1) / kUnit + item_cost(GATHER)) * (a.pool.Hkv * a.groups);
    pre[t + 1] = local;
  }
  uint64_t x = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tot[warp] = x;
  __syncthreads();
  uint64_t before = x - local;
  for (int w = 0; w < warp; ++w) before += tot[w];
  for (int t = b0; t < b1; ++t) pre[t + 1] += before;
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
}

// CTAs of an SM by registers: 128 a thread hold the state of 8 heads.  (96 and five CTAs also do without
// spills for bf16, but took 495 us for 480 us at 16 x 128K tokens.)  The kernels of fp32 queries with d = 128 spill
// 24 to 80 bytes a thread.
__host__ __device__ constexpr int resident_ctas(int HB) { return HB == 16 ? 2 : 4; }

template <int D, int NT, int SPLIT, bool GATHER>
__global__ void __launch_bounds__(kThreads, resident_ctas(8 * NT)) kv4_attn_kernel(const AttnArgs a) {
  using St = Stage<D>;
  constexpr int KS = D / 16;      // k-steps of S, and 16-row pieces of O
  constexpr int RB = D / 2;       // bytes of a code row
  constexpr int HB = 8 * NT;      // heads of an item
  constexpr uint32_t kCost = item_cost(GATHER);
  constexpr int kRing = kWarps * 2 * St::kBytes;
  constexpr int kJoin = kWarps * HB * (D + 2) * 4;
  __shared__ __align__(16) uint8_t ring[kRing > kJoin ? kRing : kJoin];
  __shared__ uint64_t pre[kMaxT + 1];
  __shared__ uint64_t tot[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  pdl_trigger();
  unit_prefix<GATHER>(a, pre, tot);
  if (blockIdx.x == 0)
    for (int t = threadIdx.x; t <= a.T; t += kThreads) a.pre[t] = pre[t];
  const uint64_t W = pre[a.T];
  const uint64_t grid = W < gridDim.x ? W : gridDim.x;
  if (blockIdx.x >= grid) return;
  uint64_t pos = W * blockIdx.x / grid;
  const uint64_t end = W * (blockIdx.x + 1) / grid;
  const int items = a.pool.Hkv * a.groups;
  uint8_t* const my_ptr = ring + warp * 2 * St::kBytes;
  const uint32_t my_ring = static_cast<uint32_t>(__cvta_generic_to_shared(my_ptr));
  const int64_t page_bytes = a.pool.page_bytes();
  const uint32_t slab_bytes = (uint32_t)a.pool.slab_bytes(), scales_at = (uint32_t)a.pool.scales_at();
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
    const uint32_t span = (uint32_t)((pre[t + 1] - pre[t]) / items), units = span - kCost;  // of one item
    const uint64_t at = pos - pre[t];
    const int item = (int)(at / span);
    const uint32_t s0 = (uint32_t)(at - (uint64_t)item * span);
    const uint32_t s1 = (uint32_t)min((uint64_t)span, s0 + (end - pos));
    pos += s1 - s0;
    if (s1 <= kCost) continue;  // nothing but the item's start
    const uint32_t u0 = s0 > kCost ? s0 - kCost : 0u, u1 = s1 - kCost;
    const int hk = item / a.groups, hg = item - hk * a.groups;
    const int nt = clamp_len(__ldg(a.n + t), a.L);
    const int len = GATHER ? a.P : nt;
    const int heads = min(HB, a.G - hg * HB);           // of this item
    const int64_t h0 = (int64_t)t * a.Hq + hk * a.G + hg * HB;

    // warp w takes steps w, w + kWarps, ... of the segment; lane l looks up row l (gathered) or the
    // first row of its half warp's piece, two steps (gathered: three) before its copy is issued
    const int p0 = (int)u0 * kUnit + warp * kTile, steps = (int)(u1 - u0);
    const uint8_t* const slab = a.pool.base + (int64_t)(2 * hk) * slab_bytes;
    const int32_t* const trow = a.pool.table + (int64_t)t * a.pool.max_pages;
    const int32_t* const irow = GATHER ? a.idx + (int64_t)t * a.P : nullptr;
    struct Row {
      int tok, page, slot;  // tok, page < 0: nothing there
    };
    auto token_of = [&](int i) -> int {
      const int p = p0 + i * kUnit + (GATHER ? lane : (lane & 16));
      if (i >= steps || p >= len) return -1;
      if (!GATHER) return p;
      const int s = __ldg(irow + p);
      count_bad_id(kBadCandidate, s != -1 && (s < 0 || s >= nt) && item == 0);
      return s >= 0 && s < nt ? s : -1;
    };
    auto row_of = [&](int tok) -> Row {
      Row w;
      w.tok = tok;
      w.page = -1;
      w.slot = 0;
      if (tok >= 0) {
        const uint32_t piece = (uint32_t)tok >> 4;  // of 16 rows; exact below 2^30 rows
        const uint32_t lp = a.page_mul ? __umulhi(piece, a.page_mul) : piece;
        w.slot = tok - (int)(lp * (uint32_t)a.pool.page_size);
        const int pg = __ldg(trow + lp);
        count_bad_id(kBadPage, (pg < 0 || pg >= a.pool.num_pages) && item == 0 && (GATHER || (lane & 15) == 0));
        w.page = pg >= 0 && pg < a.pool.num_pages ? pg : -1;
      }
      return w;
    };
    // starts the copies of one step into buffer st; returns the mask of its rows that are there
    auto issue = [&](const Row& w, int st) -> uint32_t {
      const uint32_t dst = my_ring + st * St::kBytes;
      uint32_t mask;
      if (!GATHER) {
        const int l16 = lane & 15;
        mask = __ballot_sync(0xffffffffu, w.page >= 0 && w.tok + l16 < len);
        if (w.page >= 0) {
          const uint32_t d0 = dst + (lane >> 4) * St::kPiece + l16 * 16;
          const uint8_t* page = slab + w.page * page_bytes;
          const uint8_t* ks = page + (uint32_t)(w.slot * RB + l16 * 16);
          const uint8_t* vs = ks + slab_bytes;
#pragma unroll
          for (int y = 0; y < St::kCodes / 256; ++y) copy_async<16>(d0 + y * 256, ks + y * 256);
#pragma unroll
          for (int y = 0; y < St::kCodes / 256; ++y) copy_async<16>(d0 + St::kV + y * 256, vs + y * 256);
          constexpr int SC = St::kScales / 16;  // 16-byte pieces of one side's scales
          if (l16 < 2 * SC)
            copy_async<16>(d0 + St::kKs,
                           page + (uint32_t)(scales_at + w.slot * KS + (l16 % SC) * 16) + (l16 / SC) * slab_bytes);
        }
      } else {
        mask = __ballot_sync(0xffffffffu, w.page >= 0);
        const uint8_t* page = slab + (w.page >= 0 ? w.page : 0) * page_bytes;
        const uint64_t row = reinterpret_cast<uint64_t>(page + (uint32_t)(w.slot * RB));
        constexpr int CR = RB / 16, RI = 32 / CR;  // 16-byte pieces of a code row, rows a copy covers
#pragma unroll
        for (int y = 0; y < kTile / RI; ++y) {
          const int rw = y * RI + lane / CR;
          const uint8_t* src = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, row, rw)) + lane % CR * 16;
          const uint32_t d0 = dst + (rw >> 4) * St::kPiece + (rw & 15) * RB + lane % CR * 16;
          if ((mask >> rw) & 1u) {
            copy_async<16>(d0, src);
            copy_async<16>(d0 + St::kV, src + slab_bytes);
          }
        }
        if (w.page >= 0) {
          const uint8_t* sc = page + (uint32_t)(scales_at + w.slot * KS);
          const uint32_t d0 = dst + (lane >> 4) * St::kPiece + St::kKs + (lane & 15) * KS;
          copy_async<KS>(d0, sc);
          copy_async<KS>(d0 + St::kScales, sc + slab_bytes);
        }
      }
      copy_commit();
      return mask;
    };
    Row row_next = row_of(token_of(0));
    uint32_t mask_next = issue(row_next, 0);
    row_next = row_of(token_of(1));
    int tok_next = GATHER ? token_of(2) : 0;

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

#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      const uint32_t mask = mask_next;
      copy_wait<0>();
      __syncwarp();  // the step's rows are in, and the other buffer's have been used by every lane
      if (i + 1 < steps) {
        mask_next = issue(row_next, (i + 1) & 1);
        row_next = row_of(GATHER ? tok_next : token_of(i + 2));
        if (GATHER) tok_next = token_of(i + 3);
      }
      uint8_t* sp = my_ptr + (i & 1) * St::kBytes;
      if (mask != 0xffffffffu) {
        // rows that are not there hold what the buffer held before: any codes are numbers, scales of zero
        // make them zeros
        if (!((mask >> lane) & 1u)) {
          uint8_t* z = sp + (lane >> 4) * St::kPiece + St::kKs + (lane & 15) * KS;
#pragma unroll
          for (int y = 0; y < KS / 4; ++y)
            *reinterpret_cast<uint32_t*>(z + 4 * y) = *reinterpret_cast<uint32_t*>(z + St::kScales + 4 * y) = 0u;
        }
        __syncwarp();
      }

      // S^T = K Q^T
      float s[2][NT][4];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint8_t* kp = sp + g * St::kPiece;
#pragma unroll
        for (int x = 0; x < NT; ++x) s[g][x][0] = s[g][x][1] = s[g][x][2] = s[g][x][3] = 0.f;
        uint32_t ka[KS / 2], kb[KS / 2], sa[KS / 4], sb[KS / 4];
        if constexpr (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(kp + r * RB + c * 16);
          const uint4 v = *reinterpret_cast<const uint4*>(kp + (r + 8) * RB + c * 16);
          ka[0] = u.x, ka[1] = u.y, ka[2] = u.z, ka[3] = u.w;
          kb[0] = v.x, kb[1] = v.y, kb[2] = v.z, kb[3] = v.w;
          const uint2 e = *reinterpret_cast<const uint2*>(kp + St::kKs + r * KS);
          const uint2 f = *reinterpret_cast<const uint2*>(kp + St::kKs + (r + 8) * KS);
          sa[0] = e.x, sa[1] = e.y, sb[0] = f.x, sb[1] = f.y;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(kp + r * RB + c * 8);
          const uint2 v = *reinterpret_cast<const uint2*>(kp + (r + 8) * RB + c * 8);
          ka[0] = u.x, ka[1] = u.y;
          kb[0] = v.x, kb[1] = v.y;
          sa[0] = *reinterpret_cast<const uint32_t*>(kp + St::kKs + r * KS);
          sb[0] = *reinterpret_cast<const uint32_t*>(kp + St::kKs + (r + 8) * KS);
        }
#pragma unroll
        for (int w = 0; w < KS / 2; ++w) {
          uint32_t x0[4], x1[4];
          e2m1x8_to_half2(ka[w], x0[0], x0[1], x0[2], x0[3]);
          e2m1x8_to_half2(kb[w], x1[0], x1[1], x1[2], x1[3]);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            // a block's products come out unscaled; its scale of either row goes on in fp32, as the e4m3
            // number times 2^-120 (its bits at the bottom of the exponent field; also below e4m3's normal range)
            const float ea = scale_bits(sa[w / 2], (2 * w + y) % 4), eb = scale_bits(sb[w / 2], (2 * w + y) % 4);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int z = 0; z < SPLIT; ++z)
                mma_f16(d, x0[2 * y], x1[2 * y], x0[2 * y + 1], x1[2 * y + 1], qf[z][x][2 * w + y][0],
                        qf[z][x][2 * w + y][1]);
              s[g][x][0] = fmaf(ea, d[0], s[g][x][0]);
              s[g][x][1] = fmaf(ea, d[1], s[g][x][1]);
              s[g][x][2] = fmaf(eb, d[2], s[g][x][2]);
              s[g][x][3] = fmaf(eb, d[3], s[g][x][3]);
            }
          }
        }
      }
      // logits in base 2, rows without a token minus infinity; s[g][x][0..1] row r, s[g][x][2..3] row r + 8
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) s[g][x][y] = s[g][x][y] * 0x1p120f * mul[x][y & 1];
      if (mask != 0xffffffffu) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const bool v0 = (mask >> (16 * g + r)) & 1u, v1 = (mask >> (16 * g + r + 8)) & 1u;
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            s[g][x][0] = v0 ? s[g][x][0] : -INFINITY;
            s[g][x][1] = v0 ? s[g][x][1] : -INFINITY;
            s[g][x][2] = v1 ? s[g][x][2] : -INFINITY;
            s[g][x][3] = v1 ? s[g][x][3] : -INFINITY;
          }
        }
      }
      if (a.logits) {
        const int p = p0 + i * kUnit + r;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int head = x * 8 + 2 * c + y;
            if (head < heads) {
              float* row = a.logits + (h0 + head) * a.ldS + p;
              row[0] = s[0][x][y];
              row[8] = s[0][x][2 + y];
              row[16] = s[1][x][y];
              row[24] = s[1][x][2 + y];
            }
          }
      }
      // the running maximum is raised only when a logit passes it by kSlack
      float top[NT][2];
      bool raise = false;
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          top[x][y] = fmaxf(fmaxf(s[0][x][y], s[0][x][2 + y]), fmaxf(s[1][x][y], s[1][x][2 + y]));
          raise |= top[x][y] > m[x][y] + kSlack;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float v = top[x][y];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            const float next = fmaxf(m[x][y], v);
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
      uint32_t pb[2][SPLIT][NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const float z0 = m[x][0] == -INFINITY ? 0.f : m[x][0] - kLift, z1 = m[x][1] == -INFINITY ? 0.f : m[x][1] - kLift;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float w0 = exp2_fast(s[g][x][0] - z0), w1 = exp2_fast(s[g][x][1] - z1);
          const float w2 = exp2_fast(s[g][x][2] - z0), w3 = exp2_fast(s[g][x][3] - z1);
          l[x][0] += w0 + w2;
          l[x][1] += w1 + w3;
          const uint32_t h0_ = pack_half2(w0, w1), h1_ = pack_half2(w2, w3);
          pb[g][0][x][0] = transpose8(h0_);
          pb[g][0][x][1] = transpose8(h1_);
          if (SPLIT == 2) {
            const float2 b0 = unpack_half2(h0_), b1 = unpack_half2(h1_);
            pb[g][SPLIT - 1][x][0] = transpose8(pack_half2(w0 - b0.x, w1 - b0.y));
            pb[g][SPLIT - 1][x][1] = transpose8(pack_half2(w2 - b1.x, w3 - b1.y));
          }
        }
      }

      // O^T += V^T P^T: byte i of a lane's chunk holds piece i's rows r (low nibble) and r + 8 (high)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        constexpr int W = KS / 4;  // words of a lane's chunk: 4 pieces, 2 blocks of 16 elements each
        const uint8_t* vp = sp + g * St::kPiece + St::kV + r * (RB / 8);
        const uint8_t* vs = sp + g * St::kPiece + St::kVs + (r & 1) * (KS / 2);
        uint32_t xv[4][W], ev[4];  // tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int tk = 2 * c + (y & 1) + 8 * (y >> 1);
          if constexpr (D == 128) {
            const uint2 u = *reinterpret_cast<const uint2*>(vp + tk * RB);
            xv[y][0] = u.x;
            xv[y][W - 1] = u.y;
            ev[y] = *reinterpret_cast<const uint32_t*>(vs + tk * KS);
          } else {
            xv[y][0] = *reinterpret_cast<const uint32_t*>(vp + tk * RB);
            ev[y] = *reinterpret_cast<const uint16_t*>(vs + tk * KS);
          }
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
          uint32_t lo[2][4], hi[2][4];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t xa = xv[2 * hf][w], xb = xv[2 * hf + 1][w];
            e2m1x8_to_half2((xa & 0x0f0f0f0fu) | ((xb << 4) & 0xf0f0f0f0u), lo[hf][0], lo[hf][1], lo[hf][2], lo[hf][3]);
            e2m1x8_to_half2(((xa >> 4) & 0x0f0f0f0fu) | (xb & 0xf0f0f0f0u), hi[hf][0], hi[hf][1], hi[hf][2], hi[hf][3]);
            // scales of the word's first block: a, b; of its second: a, b
            const uint32_t ab = __byte_perm(ev[2 * hf], ev[2 * hf + 1], w ? 0x7362 : 0x5140);
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
                mma_f16(o[x][4 * w + y], lo[0][y], hi[0][y], lo[1][y], hi[1][y], pb[g][z][x][0], pb[g][z][x][1]);
        }
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

// The pieces of a (query, head): count 0 where it attends to nothing, 1 where one CTA had it whole (and has
// written its output and log-sum), else the pieces lie in slots first, first + 1, ...
struct Pieces {
  int64_t first;
  int count;
};

__device__ __forceinline__ Pieces pieces_of(const AttnArgs& a, int t, int hq, int HB, int64_t ctas) {
  const int hk = hq / a.G, hr = hq % a.G;
  const int items = a.pool.Hkv * a.groups, item = hk * a.groups + hr / HB;
  const uint64_t W = a.pre[a.T], first = a.pre[t];
  const uint64_t span = (a.pre[t + 1] - first) / items;
  Pieces r = {0, 0};
  if (span > 0) {
    const uint64_t grid = W < (uint64_t)ctas ? W : (uint64_t)ctas;
    const uint64_t p0 = first + item * span + item_cost(a.idx != nullptr), p1 = first + (item + 1) * span;
    const int64_t c0 = (int64_t)(((p0 + 1) * grid - 1) / W), c1 = (int64_t)((p1 * grid - 1) / W);
    r.first = c0 + (int64_t)t * items + item;
    r.count = (int)(c1 - c0 + 1);
  }
  return r;
}

__device__ __forceinline__ float2 piece_ml(const AttnArgs& a, int64_t slot, int HB, int head) {
  return *reinterpret_cast<const float2*>(a.part_ml + (slot * HB + head) * 2);
}

template <int SPLIT>
__device__ __forceinline__ void store_out(const AttnArgs& a, int64_t at, float v) {
  if (SPLIT == 1) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
  else static_cast<float*>(a.out)[at] = v;
}

__device__ __forceinline__ void store_lse(const AttnArgs& a, int64_t hd, float top, float sum) {
  const float z = sum == 0.f ? -INFINITY : top + log2f(sum) - kLift;
  if (a.lse) a.lse[hd] = z * 0.693147180559945309f;
  if (a.lse2) a.lse2[hd] = z;
}

// The joins of one head by a whole CTA: its threads first weigh the pieces (each by its maximum against the
// largest), then its warps add up every eighth piece.
template <int D, int SPLIT>
__device__ __forceinline__ void join_wide(const AttnArgs& a, int hd, int HB, int64_t ctas) {
  constexpr int E = D / 32;  // output elements of a lane
  __shared__ float weight[kMaxCtas];
  __shared__ float red[8];
  __shared__ __align__(16) float part[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = hd / a.Hq, hq = hd % a.Hq, head = hq % a.G % HB;
  const Pieces pc = pieces_of(a, t, hq, HB, ctas);
  if (pc.count == 1) return;
  auto over_block = [&](float v, bool largest) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float w = __shfl_xor_sync(0xffffffffu, v, o);
      v = largest ? fmaxf(v, w) : v + w;
    }
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) v = largest ? fmaxf(v, red[w]) : v + red[w];
    return v;
  };
  constexpr int kPer = kMaxCtas / 256;
  float2 ml[kPer];
  float top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int i = x * 256 + threadIdx.x;
    ml[x] = i < pc.count ? piece_ml(a, pc.first + i, HB, head) : make_float2(-INFINITY, 0.f);
    top = fmaxf(top, ml[x].x);
  }
  top = over_block(top, true);
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int i = x * 256 + threadIdx.x;
    const float f = ml[x].y == 0.f ? 0.f : exp2_fast(ml[x].x - top);
    if (i < pc.count) weight[i] = f;
    sum += f * ml[x].y;
  }
  sum = over_block(sum, false);
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int i = warp; i < pc.count; i += 8) {
    const float* p = a.part + ((pc.first + i) * HB + head) * D + lane * E;
    const float f = weight[i];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += f * p[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += part[w][threadIdx.x];
    store_out<SPLIT>(a, (int64_t)hd * D + threadIdx.x, v * (sum == 0.f ? 0.f : a.v_scale / sum));
  }
  if (threadIdx.x == 0) store_lse(a, hd, top, sum);
}

// The join of one head by a warp.
template <int D, int SPLIT>
__device__ __forceinline__ void join_narrow(const AttnArgs& a, int hd, int HB, int64_t ctas) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, t = hd / a.Hq, hq = hd % a.Hq, head = hq % a.G % HB;
  const Pieces pc = pieces_of(a, t, hq, HB, ctas);
  if (pc.count == 1) return;
  float top = -INFINITY, sum = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i = lane; i < pc.count; i += 32) top = fmaxf(top, piece_ml(a, pc.first + i, HB, head).x);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 4
  for (int i = 0; i < pc.count; ++i) {
    const float2 ml = piece_ml(a, pc.first + i, HB, head);
    const float* p = a.part + ((pc.first + i) * HB + head) * D + lane * E;
    const float f = ml.y == 0.f ? 0.f : exp2_fast(ml.x - top);
    sum += f * ml.y;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += f * p[e];
  }
  const float inv = sum == 0.f ? 0.f : a.v_scale / sum;
#pragma unroll
  for (int e = 0; e < E; ++e) store_out<SPLIT>(a, (int64_t)hd * D + lane * E + e, acc[e] * inv);
  if (lane == 0) store_lse(a, hd, top, sum);
}

// Joins the pieces of a (query, head) whose tokens more than one CTA took; also writes the heads of queries that
// attend to nothing.  WIDE: a CTA a head, else a warp.
template <int D, int SPLIT, bool WIDE>
__global__ void __launch_bounds__(256) kv4_join_kernel(const AttnArgs a, int HB, int64_t ctas) {
  pdl_wait();
  if (WIDE) {
    join_wide<D, SPLIT>(a, blockIdx.x, HB, ctas);
  } else {
    const int hd = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (hd < a.T * a.Hq) join_narrow<D, SPLIT>(a, hd, HB, ctas);
  }
}

// acc[t, i] += sum over the heads of token i's weight, i < cols, from the logits and every head's log-sum.  SHARE threads
// a position, each every SHARE-th head, and their sums in order.
// Selected tokens are added atomically: a token that a list names twice gets both of its (equal)
// weights, in either order the same sum.
template <int SHARE>
__global__ void __launch_bounds__(256)
    kv4_weights_kernel(const AttnArgs a, float* __restrict__ acc, int cols, int64_t ld) {
  constexpr int kTokens = 256 / SHARE;
  __shared__ float part[SHARE][kTokens];
  pdl_wait();
  const int t = blockIdx.y, nt = clamp_len(__ldg(a.n + t), a.L);
  const int x = threadIdx.x % kTokens, y = threadIdx.x / kTokens, p = blockIdx.x * kTokens + x;
  int s = p < (a.idx ? a.P : nt) ? p : -1;
  if (a.idx && s >= 0) s = __ldg(a.idx + (int64_t)t * a.P + p);
  const bool there = s >= 0 && s < min(nt, cols);
  float w = 0.f;
  if (there) {
    const float* row = a.logits + (int64_t)t * a.Hq * a.ldS + p;
    const float* z = a.lse2 + (int64_t)t * a.Hq;
#pragma unroll (SHARE == 1 ? 8 : 16)
    for (int h = y; h < a.Hq; h += SHARE) {
      const float lz = z[h], v = row[h * a.ldS];
      w += lz == -INFINITY ? 0.f : exp2_fast(v - lz);
    }
  }
  if (SHARE > 1) {
    part[y][x] = w;
    __syncthreads();
    if (y != 0) return;
    w = part[0][x];
#pragma unroll
    for (int i = 1; i < SHARE; ++i) w += part[i][x];
  }
  if (!there) return;
  float* dst = acc + (int64_t)t * ld + s;
  if (a.idx) atomicAdd(dst, w);
  else *dst += w;
}

int heads_per_item(int G) { return G > 8 ? 16 : 8; }

int64_t attn_ctas(int T, int P, int Hkv, int G, bool selected) {
  const int HB = heads_per_item(G);
  const int64_t most = (int64_t)T * Hkv * ((G + HB - 1) / HB) * ((P + kUnit - 1) / kUnit + item_cost(selected));
  const int64_t full = std::min<int64_t>((int64_t)sm_count() * resident_ctas(HB), kMaxCtas);
  return std::min(most, full);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <int D, int NT, int SPLIT>
void launch_attn(const AttnArgs& a, float* acc, int cols, int64_t ld_acc, int64_t ctas, cudaStream_t s) {
  if (ctas > 0) {
    if (a.idx) kv4_attn_kernel<D, NT, SPLIT, true><<<(unsigned)ctas, kThreads, 0, s>>>(a);
    else kv4_attn_kernel<D, NT, SPLIT, false><<<(unsigned)ctas, kThreads, 0, s>>>(a);
  }
  // A CTA a head where a wave of them is enough (a warp each is slower by 2 us) or where the pieces are many (74 of
  // them, 16K tokens of one sequence, took a warp 25 us), else a warp: 2048 heads of 5 pieces 6 us for 11.
  const int heads = a.T * a.Hq;
  const bool wide = heads <= 148 * 4 || ctas > 16 * (int64_t)(a.T * a.pool.Hkv * a.groups);
  if (wide) launch_pdl(kv4_join_kernel<D, SPLIT, true>, dim3(heads), dim3(256), 0, s, a, 8 * NT, ctas);
  else launch_pdl(kv4_join_kernel<D, SPLIT, false>, dim3((heads + 7) / 8), dim3(256), 0, s, a, 8 * NT, ctas);
  if (acc) {
    // few positions do not fill the GPU with a thread each: 32 x 2048 selected ones take 9 us for 15 with four;
    // 32 x 16384 take 10 us, with four 14
    auto weights = [&](auto kernel, int tokens) {
      launch_pdl(kernel, dim3((a.P + tokens - 1) / tokens, a.T), dim3(256), 0, s, a, acc, cols, ld_acc);
    };
    if ((int64_t)a.T * a.P <= 148 * 1024) weights(kv4_weights_kernel<4>, 64);
    else weights(kv4_weights_kernel<1>, 256);
  }
}

// Positions that a query's logits have room for.
int64_t logit_row(int P) { return ((int64_t)P + kUnit - 1) / kUnit * kUnit; }

// Queries of a launch.
int queries_per_launch(int T, int P, int Hq, bool weights) {
  int64_t most = kMaxT;
  if (weights) most = std::min<int64_t>(most, std::max<int64_t>(1, kLogitBytes / (sizeof(float) * Hq * logit_row(P))));
  return (int)std::min<int64_t>(T, most);
}

}  // namespace

size_t kv4_attention_ws_bytes(int T, int P, int Hq, int Hkv, int d, bool weights) {
  const int G = Hq / Hkv, HB = heads_per_item(G);
  const int Tc = queries_per_launch(T, P, Hq, weights);
  const int64_t slots = kMaxCtas + (int64_t)Tc * Hkv * ((G + HB - 1) / HB);
  size_t b = up256(sizeof(uint64_t) * (kMaxT + 1)) + up256(sizeof(float) * slots * HB * d) +
             up256(sizeof(float) * slots * HB * 2);
  if (weights)
    b += up256(sizeof(float) * (size_t)Tc * Hq) +
         up256(sizeof(float) * (size_t)Tc * Hq * logit_row(P));
  return b;
}

void launch_kv4_attention(DType dt, const void* q, const Kv4Pool& pool, const int32_t* n, const int32_t* idx, int T,
                          int L, int P, int Hq, float scale, float k_scale, float v_scale, void* out, float* lse,
                          float* acc, int acc_cols, int64_t ld_acc, void* ws, cudaStream_t s) {
  const int G = Hq / pool.Hkv, HB = heads_per_item(G);
  const size_t elt = dt == DType::BF16 ? 2 : 4;
  const int most = queries_per_launch(T, P, Hq, acc != nullptr);
  for (int t0 = 0; t0 < T; t0 += most) {
    const int Tc = std::min(T - t0, most);
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
    const uint32_t pieces = (uint32_t)pool.page_size / kSub;
    a.page_mul = pieces == 1 ? 0u : (uint32_t)(((1ull << 32) + pieces - 1) / pieces);
    a.out = static_cast<char*>(out) + elt * t0 * (size_t)Hq * pool.d;
    a.lse = lse ? lse + (int64_t)t0 * Hq : nullptr;
    const int64_t ctas = attn_ctas(Tc, a.P, pool.Hkv, G, idx != nullptr);
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
      a.ldS = logit_row(a.P);
      ac = acc + (int64_t)t0 * ld_acc;
    }
    const bool f32 = dt == DType::F32;
    auto run = [&](auto launch) { launch(a, ac, acc_cols, ld_acc, ctas, s); };
    if (pool.d == 128) {
      if (HB == 8) f32 ? run(launch_attn<128, 1, 2>) : run(launch_attn<128, 1, 1>);
      else f32 ? run(launch_attn<128, 2, 2>) : run(launch_attn<128, 2, 1>);
    } else {
      if (HB == 8) f32 ? run(launch_attn<64, 1, 2>) : run(launch_attn<64, 1, 1>);
      else f32 ? run(launch_attn<64, 2, 2>) : run(launch_attn<64, 2, 1>);
    }
  }
}

MISA_BAD_ID_READER(read_and_clear_bad_ids_kv4_attn)

}  // namespace misa
