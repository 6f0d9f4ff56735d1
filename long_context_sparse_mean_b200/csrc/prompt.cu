// Causal attention of packed prompts with grouped heads:
//   out_{i,h} = sum_{j <= i + o_b} softmax_j(scale q_{i,h} . k_{j,h'}) v_{j,h'},   o_b = keys - queries of b
// so the queries of a sequence are its last ones (o_b > 0 when earlier keys come from a cache), and a
// query with nothing to see (o_b < 0) gets zeros and a log-sum of minus infinity.
//
// What bounds it: 4 d operations for every (query, key, head) pair that is seen, on the tensor cores
// (4096 multiply-adds a clock and SM), and as much time again for the pair's exponential (16 a clock and
// SM): a 128 x 128 piece takes 2 x 512 clocks of products at d = 128 and 1024 of exponentials.  So a CTA
// works on two tiles of 128 queries at once: while one tile's scores go through the softmax, the tensor
// cores multiply for the other.
//
// Per CTA (one per SM): 256 queries of one head, tiles A and B, and the keys they see in ascending
// blocks of 128.  S = Q K^T and O += P V run on tcgen05 with fp32 accumulators in tensor memory
// (S_A, S_B, O_A, O_B: 128 columns each, all 512); P overwrites the first half of its S as bf16, the A
// operand of the second product.  Warp roles:
//   warps 0-3, 4-7  softmax of tile A, B: one thread a query row, so row maxima and sums need no
//                   exchange; also rescale O, normalise and write the output
//   warp 8          TMA producer: the two Q tiles, then K and V blocks through a ring of buffers
//   warp 9          MMA issuer (one thread) and owner of the tensor memory
//   warps 10, 11    guards: in the blocks where some query does not see every key they set to zero the
//                   value rows behind the sequence and every value that is not finite (a weight of
//                   zero times such a value would not be zero), before the product reads them
// The running maximum m is raised, and O rescaled, only when a row's scores pass it by 8 (base 2): O and
// the sum stay right for any m, and weights up to 2^8 lose nothing in bf16 or fp32.  Weights are rounded
// to bf16 (2^-9) for the product with V, of the same type; their sum is taken before, in fp32.
// Values that are not finite and were set to zero are added to the rows that do see them at the end.
// Every wait is bounded in time; a wait that runs out sets a device status word and all roles leave
// their loops, wait for their own copies and MMAs, and free tensor memory.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstring>

#include "kernels.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace misa {

namespace {

// Nonzero after the kernel gave up on a wait (read and cleared by misa_device_check).
__device__ int g_prompt_status = 0;

constexpr int kRows = 128;                  // queries of a tile, keys of a block
constexpr int kPair = 2 * kRows;            // queries of a CTA
constexpr int kThreads = 12 * 32;
// Registers a thread: 384 threads launch with 168 (64512 in all); 256 x 200 + 128 x 104 is the same.
constexpr int kRegsSoftmax = 200, kRegsOther = 104;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= 168 * kThreads, "register split exceeds the launch's registers");
constexpr int kLoadWarp = 8, kMmaWarp = 9, kGuardWarp = 10;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // 1 s
constexpr int kLag = 6;                     // pairs of weights between their exponentials and their sum
constexpr float kSlack = 8.f;               // base-2 growth of a row's scores before its maximum is raised

template <int D>
struct Lay {
  static constexpr int kTileBytes = kRows * D * 2;         // one Q tile, K block or V block
  static constexpr int kHalfBytes = kRows * 64 * 2;        // 64 dimensions of it (one swizzled box)
  static constexpr int kBufs = D == 128 ? 4 : 8;           // ring of K and V blocks
  static constexpr int kOffQ = 0;
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kOffBar = kOffRing + kBufs * kTileBytes;
  static constexpr int kNumBars = 2 + 3 * kBufs + 8 + 1;
  static constexpr int kOffMisc = kOffBar + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kSmem = kOffMisc + 256 + 1024;      // + alignment slack
};

struct PromptArgs {
  const __nv_bfloat16* v;
  int64_t ldv;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int S, Tq, Tk, Hq, G;
  float c;                // scale times log2(e)
  __nv_bfloat16* out;
  float* lse;
};

// What a CTA works on: rows [row, row + rows) of the queries, `keys` keys from key0 on; query i of the
// pair sees keys j <= i + off.
struct Item {
  int row, rows, key0, keys, off, head;
  // blocks that tile t (0, 1) reads
  __device__ __forceinline__ int blocks(int t) const {
    if (t * kRows >= rows) return 0;
    const int last = min(keys, min((t + 1) * kRows, rows) + off);  // keys seen by the tile's last row
    return last > 0 ? (last + kRows - 1) / kRows : 0;
  }
  // whether some query of tile t does not see all keys of block j
  __device__ __forceinline__ bool masked(int t, int j) const {
    const int end = (j + 1) * kRows;
    return end > keys || end - 1 > t * kRows + off;
  }
};

// Waits for the barrier phase with this parity; false once *abort is set or after the time limit.  The
// clock and the abort word are looked at every 256 tries only: reading the clock takes about as long
// as a piece of the softmax.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, const volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t spin = 1;; ++spin) {
    if (tc::mbar_test(bar, parity)) return true;
    if ((spin & 255u) == 0) {
      if (abort && *abort) return false;
      const uint64_t now = tc::global_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) return false;
    }
  }
}

__device__ __forceinline__ void give_up(volatile int* abort) {
  *abort = 1;
  atomicExch(&g_prompt_status, 1);
}

// True in one thread of the warp, chosen so that the compiler knows there is only one (tensor-core and bulk
// copy instructions take warp-uniform operands; under a test of the lane number it loops over lanes).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// Shared-memory descriptor of V [keys][64 dims] boxes as the B operand with dims contiguous: 64-element
// columns of 8-key atoms (1024 bytes) under the 128-byte swizzle, the next 64 dims kHalfBytes on.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t lead) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// D[tmem] (+)= A[tmem] * B[smem], issued by one thread.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Scores from position `seen` on become minus infinity.
__device__ __forceinline__ void hide(uint32_t (&s)[32], int seen) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (e >= seen) s[e] = 0xff800000u;
}

// Warp-wide: lane l writes 16 consecutive columns of TMEM lane (taddr.lane + l).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Warp-wide: lane l writes 32 consecutive columns of TMEM lane (taddr.lane + l).
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The item of CTA x: pairs of every sequence from its last to its first (the longest come first), the
// heads of a pair next to each other.  False when there is none.  Every thread of the block calls it.
__device__ __forceinline__ bool find_item(const PromptArgs& a, int x, Item& it, uint32_t* warp_tot, int* found) {
  const int pair = x / a.Hq;
  it.head = x - pair * a.Hq;
  int base = 0;
  if (threadIdx.x == 0) found[0] = -1;
  for (int b0 = 0; b0 < a.S; b0 += kThreads) {
    const int b = b0 + (int)threadIdx.x;
    int q0 = 0, m = 0;
    if (b < a.S) {
      q0 = max(0, __ldg(a.cu_q + b));
      m = max(0, min(a.Tq, __ldg(a.cu_q + b + 1)) - q0);
    }
    const int tiles = (m + kPair - 1) / kPair;
    uint32_t total;
    const int before = base + (int)block_exclusive_scan((uint32_t)tiles, warp_tot, &total);
    if (pair >= before && pair < before + tiles) {
      const int t = tiles - 1 - (pair - before);
      const int k0 = max(0, __ldg(a.cu_k + b)), k1 = min(a.Tk, __ldg(a.cu_k + b + 1));
      const int l = max(0, k1 - k0);
      found[0] = q0 + t * kPair;
      found[1] = min(kPair, m - t * kPair);
      found[2] = k0;
      found[3] = l;
      found[4] = l - m + t * kPair;
    }
    __syncthreads();
    if (found[0] >= 0) break;
    base += (int)total;
    if (base > pair) break;
  }
  if (a.S <= 0 || found[0] < 0) return false;
  it.row = found[0];
  it.rows = found[1];
  it.key0 = found[2];
  it.keys = found[3];
  it.off = found[4];
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const PromptArgs a) {
  using L = Lay<D>;
  constexpr int NB = L::kBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + L::kOffMisc);
  volatile uint32_t* tmem_slot = misc;
  volatile int* abort = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* odd = reinterpret_cast<volatile int*>(misc + 2);  // a value that is not finite was set to zero
  int* found = reinterpret_cast<int*>(misc + 4);
  uint32_t* warp_tot = misc + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  Item it;
  if (!find_item(a, blockIdx.x, it, warp_tot, found)) return;
  const int nA = it.blocks(0), nB = it.blocks(1), nblk = max(nA, nB);

  const uint32_t bar0 = tc::smem_u32(sm + L::kOffBar);
  auto qfull = [&](int t) { return bar0 + 8 * t; };
  auto full = [&](int i) { return bar0 + 8 * (2 + i); };
  auto empty = [&](int i) { return bar0 + 8 * (2 + NB + i); };
  auto vok = [&](int i) { return bar0 + 8 * (2 + 2 * NB + i); };
  auto sfull = [&](int t) { return bar0 + 8 * (2 + 3 * NB + t); };
  auto pfull = [&](int t) { return bar0 + 8 * (4 + 3 * NB + t); };
  auto odone = [&](int t) { return bar0 + 8 * (6 + 3 * NB + t); };
  auto phalf = [&](int t) { return bar0 + 8 * (8 + 3 * NB + t); };
  const uint32_t drain = bar0 + 8 * (10 + 3 * NB);
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(qfull(t), 1);
      tc::mbar_init(sfull(t), 1);
      tc::mbar_init(pfull(t), 4);
      tc::mbar_init(phalf(t), 4);
      tc::mbar_init(odone(t), 1);
    }
    for (int i = 0; i < NB; ++i) {
      tc::mbar_init(full(i), 1);
      tc::mbar_init(empty(i), 1);
      tc::mbar_init(vok(i), 2);
    }
    tc::mbar_init(drain, 1);
    *abort = 0;
    *odd = 0;
    tc::mbar_init_fence();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tc::smem_u32((const void*)tmem_slot), kTmemCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t qbase = tc::smem_u32(sm + L::kOffQ), ring = tc::smem_u32(sm + L::kOffRing);
  // block j's K is ring use 2 j, its V use 2 j + 1
  auto guarded = [&](int j) { return (j < nA && it.masked(0, j)) || (j < nB && it.masked(1, j)); };

  if (warp < 8) {
    // ---------------- softmax ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, n = t ? nB : nA;
    const int i = t * kRows + (warp & 3) * 32 + lane;  // query of the pair
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * kRows, to = tmem + lanes + 2 * kRows + t * kRows;
    const float c = a.c;
    float m = -INFINITY, l = 0.f;  // maximum of the raw scores, sum of the weights
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!wait_for(sfull(t), j & 1, abort)) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int x = 0; x < 4; ++x) tc::tmem_ld32(ts + 32 * x, s[x]);
#pragma unroll
      for (int x = 0; x < 4; ++x) tc::tmem_ld_wait(s[x]);
      if (it.masked(t, j)) {
        const int seen = min(it.keys, i + it.off + 1) - j * kRows;  // keys of this block that row i sees
#pragma unroll
        for (int x = 0; x < 4; ++x) hide(s[x], seen - 32 * x);
      }
      // Weights go pair by pair through multiply-add, exponential, and kLag pairs later sum and rounding, so
      // that the exponentials (8 clocks a warp and instruction) never wait for their own results; 16 pairs
      // are written at a time, over scores that have been read.  They start from the running maximum as it
      // is, while the block's own maximum is found among the first 16 pairs' exponentials; should that pass
      // it, these pairs are done again.
      float2 sum[2], w[kLag];
      uint32_t p[16];
      float neg = m == -INFINITY ? 0.f : -m * c;
      sum[0] = sum[1] = make_float2(0.f, 0.f);
      auto start = [&](int e) {  // exponentials of pair e
        const float2 z = __ffma2_rn(make_float2(__uint_as_float(s[e / 16][2 * (e % 16)]), __uint_as_float(s[e / 16][2 * (e % 16) + 1])),
                                    make_float2(c, c), make_float2(neg, neg));
        w[e % kLag] = make_float2(ex2(z.x), ex2(z.y));
      };
      auto finish = [&](int e) {  // its sum and its rounding
        const float2 v = w[e % kLag];
        sum[e & 1] = __fadd2_rn(sum[e & 1], v);
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
        p[e & 15] = *reinterpret_cast<const uint32_t*>(&h);
      };
      float top[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) top[x] = __uint_as_float(s[x][0]);
#pragma unroll
      for (int e = 0; e < 16 + kLag; ++e) {
        if (e >= kLag) finish(e - kLag);
        if (e < 16) {
          start(e);
#pragma unroll
          for (int x = 0; x < 4; ++x) top[x] = max3(top[x], __uint_as_float(s[x][2 * e]), __uint_as_float(s[x][2 * e + 1]));
        }
      }
      const float mx = max3(fmaxf(top[0], top[1]), top[2], top[3]);
      const bool raise = mx * c > m * c + kSlack;  // also the first score that is seen
      if (__any_sync(0xffffffffu, raise)) {
        if (j > 0) {
          // O holds blocks 0 .. j - 1 once their product is through
          if (!wait_for(odone(t), (j - 1) & 1, abort)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const float f = raise && m != -INFINITY ? ex2((m - mx) * c) : 1.f;
          l *= f;
#pragma unroll 1
          for (int x = 0; x < D / 32; ++x) {
            uint32_t o[32];
            tc::tmem_ld32(to + 32 * x, o);
            tc::tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(to + 32 * x, o);
          }
        }
        if (raise) m = mx;
        neg = m == -INFINITY ? 0.f : -m * c;
        sum[0] = sum[1] = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 16 + kLag; ++e) {
          if (e >= kLag) finish(e - kLag);
          if (e < 16) start(e);
        }
      }
      tmem_st16(ts, p);
#pragma unroll
      for (int e = 16; e < 64 + kLag; ++e) {
        if (e >= 16 + kLag) {
          const int y = e - kLag;
          finish(y);
          if ((y & 15) == 15) tmem_st16(ts + y - 15, p);
          if (y == 31) {  // half of the weights are there: their product may start
            tmem_st_wait();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_relaxed(phalf(t));
          }
        }
        if (e < 64) start(e);
      }
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_relaxed(pfull(t));  // what it hands on lies in tensor memory
    }
    if (ok && n > 0 && !wait_for(odone(t), (n - 1) & 1, abort)) ok = false;
    tc::tc_fence_after();
    if (!ok) give_up(abort);
    if (ok && t * kRows < it.rows) {
      const int64_t row = (int64_t)it.row + i;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      // this warp's 32 rows go through its share of the Q tile, which the products have read
      uint8_t* stage = sm + L::kOffQ + t * L::kTileBytes + (warp & 3) * 32 * D * 2;
      constexpr int CH = D / 8;  // 16-byte pieces of a row
#pragma unroll 1
      for (int x = 0; x < D / 32; ++x) {
        uint32_t o[32];
        if (n > 0) {
          tc::tmem_ld32(to + 32 * x, o);
          tc::tmem_ld_wait(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (*odd) {  // values that are not finite and that this row sees, in the blocks they were taken out of
          const int end = min(it.keys, i + it.off + 1);
          for (int j = 0; j < n; ++j) {
            if (!guarded(j)) continue;
            for (int k = j * kRows; k < min(end, (j + 1) * kRows); ++k) {
              const __nv_bfloat16* vr = a.v + (int64_t)(it.key0 + k) * a.ldv + (it.head / a.G) * D + 32 * x;
              for (int e = 0; e < 32; ++e) {
                const float f = __bfloat162float(vr[e]);
#pragma unroll
                for (int y = 0; y < 32; ++y)
                  if (y == e && !isfinite(f)) o[y] = __float_as_uint(__uint_as_float(o[y]) + f);
              }
            }
          }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(o[8 * y + 2 * e]) * inv,
                                                           __uint_as_float(o[8 * y + 2 * e + 1]) * inv);
            w[e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          const int piece = 4 * x + y;
          *reinterpret_cast<uint4*>(stage + lane * (D * 2) + ((piece ^ (lane & (CH - 1))) * 16)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
      constexpr int RPI = 32 / CH;  // rows a store instruction covers
      const int first = t * kRows + (warp & 3) * 32;
#pragma unroll 4
      for (int y = 0; y < 32; y += RPI) {
        const int rr = y + lane / CH, piece = lane % CH;
        if (first + rr < it.rows)
          *reinterpret_cast<uint4*>(a.out + ((int64_t)(it.row + first + rr) * a.Hq + it.head) * D + piece * 8) =
              *reinterpret_cast<const uint4*>(stage + rr * (D * 2) + ((piece ^ (rr & (CH - 1))) * 16));
      }
      if (a.lse && i < it.rows)
        a.lse[row * a.Hq + it.head] = l == 0.f ? -INFINITY : m * c * 0.693147180559945309f + logf(l);
    }
  } else {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  if (warp == kLoadWarp) {
    // ---------------- TMA producer ----------------
    if (elect_one()) {
      const int hk = it.head / a.G;
      bool ok = true;
      uint32_t u = 0;
      auto q_tile = [&](int t) {
        tc::mbar_arrive_expect_tx(qfull(t), L::kTileBytes);
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          tc::tma_load_2d(qbase + t * L::kTileBytes + x * L::kHalfBytes, &qmap, it.head * D + x * 64,
                          it.row + t * kRows, qfull(t));
      };
      if (nA > 0) q_tile(0);
      for (int j = 0; ok && j < nblk; ++j) {
        for (int side = 0; side < 2; ++side, ++u) {
          const int b = u % NB;
          if (u >= NB && !wait_for(empty(b), ((u / NB) - 1) & 1, abort)) {
            ok = false;
            break;
          }
          tc::mbar_arrive_expect_tx(full(b), L::kTileBytes);
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            tc::tma_load_2d(ring + b * L::kTileBytes + x * L::kHalfBytes, side ? &vmap : &kmap, hk * D + x * 64,
                            it.key0 + j * kRows, full(b));
          if (j == 0 && side == 0 && nB > 0) q_tile(1);
        }
      }
      if (!ok) give_up(abort);
      // every issued copy lands before the CTA exits
      if (nA > 0) wait_for(qfull(0), 0, nullptr);
      if (nB > 0) wait_for(qfull(1), 0, nullptr);
      for (uint32_t g = u > NB ? u - NB : 0; g < u; ++g) wait_for(full(g % NB), (g / NB) & 1, nullptr);
    }
  } else if (warp == kMmaWarp) {
    // ---------------- MMA issuer ----------------
    if (elect_one()) {
      constexpr uint32_t idesc_s = tc::idesc_bf16_f32(kRows, kRows);
      constexpr uint32_t idesc_o = tc::idesc_bf16_f32(kRows, D) | (1u << 16);  // V with its dims contiguous
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok && !wait_for(bar, parity, abort)) ok = false;
        return ok;
      };
      auto scores = [&](int t, int j) {  // S_t = Q_t K_j^T
        const uint32_t u = 2 * j, b = u % NB;
        if (j == 0 && !wait(qfull(t), 0)) return;
        if (!wait(full(b), (u / NB) & 1)) return;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t at = (kk / 4) * L::kHalfBytes + (kk % 4) * 32;
          tc::mma_bf16(tmem + t * kRows, tc::sw128_kmajor_desc(qbase + t * L::kTileBytes + at),
                       tc::sw128_kmajor_desc(ring + b * L::kTileBytes + at), idesc_s, kk != 0);
        }
        tc::mma_commit(sfull(t));
        if (t == 1 || j >= nB) tc::mma_commit(empty(b));
      };
      auto values = [&](int t, int j) {  // O_t += P_t V_j
        const uint32_t u = 2 * j + 1, b = u % NB;
        if (!wait(vok(b), (u / NB) & 1)) return;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!wait(half ? pfull(t) : phalf(t), j & 1)) return;
          tc::tc_fence_after();  // after the weights' stores to tensor memory, by other threads
#pragma unroll
          for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
            mma_bf16_ts(tmem + 2 * kRows + t * kRows, tmem + t * kRows + kk * 8,
                        sw128_mnmajor_desc(ring + b * L::kTileBytes + kk * 2048, L::kHalfBytes), idesc_o,
                        (j | kk) != 0);
        }
        tc::mma_commit(odone(t));
        if (t == 1 || j >= nB) tc::mma_commit(empty(b));
      };
      if (nA > 0) scores(0, 0);
      if (nB > 0 && ok) scores(1, 0);
      for (int j = 0; ok && j < nblk; ++j) {
        for (int t = 0; ok && t < 2; ++t) {
          const int n = t ? nB : nA;
          if (j < n) values(t, j);
          if (ok && j + 1 < n) scores(t, j + 1);
        }
      }
      if (!ok) give_up(abort);
      // every issued MMA completes before tensor memory is freed
      tc::mma_commit(drain);
      wait_for(drain, 0, nullptr);
    }
  } else {
    // ---------------- guards ----------------
    bool ok = true;
    for (int j = 0; ok && j < nblk; ++j) {
      const uint32_t u = 2 * j + 1, b = u % NB;
      if (!wait_for(full(b), (u / NB) & 1, abort)) {
        ok = false;
        break;
      }
      if (!guarded(j)) {  // passed on all the same: a guard that fell behind by a turn of the ring would miss its phase
        if (lane == 0) tc::mbar_arrive(vok(b));
        continue;
      }
      const int there = it.keys - j * kRows;  // rows from here on belong to no key of the sequence
      const int first = (warp - kGuardWarp) * (kRows / 2);
      uint8_t* v = sm + L::kOffRing + b * L::kTileBytes;
      bool changed = false, bad = false;
#pragma unroll 4
      for (int x = lane; x < (kRows / 2) * (D / 8); x += 32) {
        const int half = x / (kRows / 2 * 8), y = x % (kRows / 2 * 8);  // 8 pieces of 16 bytes a row and half
        const int r = first + y / 8;
        uint4* p = reinterpret_cast<uint4*>(v + half * L::kHalfBytes + r * 128 + (y % 8) * 16);
        if (r >= there) {
          *p = make_uint4(0u, 0u, 0u, 0u);
          changed = true;
          continue;
        }
        const uint4 w = *p;
        // a half whose exponent is all ones carries into its top bit
        auto hit = [](uint32_t z) { return ((z & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
        if (hit(w.x) | hit(w.y) | hit(w.z) | hit(w.w)) {
          auto clean = [&](uint32_t z) {
            const uint32_t h = hit(z);
            return z & ~((h >> 15) * 0xffffu);
          };
          *p = make_uint4(clean(w.x), clean(w.y), clean(w.z), clean(w.w));
          changed = bad = true;
        }
      }
      if (bad) *odd = 1;
      if (changed) tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(vok(b));
    }
    if (!ok) give_up(abort);
  }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Map over packed rows [rows][cols] of bf16 at a stride of ld elements, boxes of 64 columns x 128 rows in
// the 128-byte swizzled layout; rows past the end read as zero.
bool row_map(CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t ld) {
  const EncodeTiledFn encode = tmap_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, kRows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
bool launch_d(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const PromptArgs& a,
              cudaStream_t s) {
  static_assert(Lay<D>::kSmem <= 232448, "shared memory of the prompt kernel exceeds 227 KB");
  const int64_t grid = ((int64_t)a.Tq / kPair + std::min<int64_t>(a.S, a.Tq)) * a.Hq;
  if (grid > INT32_MAX) return false;
  cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kSmem);
  prompt_kernel<D><<<(unsigned)grid, kThreads, Lay<D>::kSmem, s>>>(qm, km, vm, a);
  return true;
}

}  // namespace

bool launch_prompt_attention(const void* q, const void* k, const void* v, int64_t ldq, int64_t ldk, int64_t ldv,
                             const int32_t* cu_q, const int32_t* cu_k, int S, int Tq, int Tk, int Hq, int Hkv, int d,
                             float scale, void* out, float* lse, cudaStream_t s) {
  if (S <= 0 || Tq <= 0) return true;
  CUtensorMap qm, km, vm;
  if (!row_map(&qm, q, (int64_t)Hq * d, Tq, ldq)) return false;
  // without keys nothing is loaded through the other two
  if (Tk <= 0) km = vm = qm;
  else if (!row_map(&km, k, (int64_t)Hkv * d, Tk, ldk) || !row_map(&vm, v, (int64_t)Hkv * d, Tk, ldv)) return false;
  PromptArgs a;
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.ldv = ldv;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.S = S;
  a.Tq = Tq;
  a.Tk = Tk;
  a.Hq = Hq;
  a.G = Hq / Hkv;
  a.c = scale * 1.44269504088896341f;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  return d == 128 ? launch_d<128>(qm, km, vm, a, s) : launch_d<64>(qm, km, vm, a, s);
}

int read_and_clear_prompt_status() {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_prompt_status, sizeof(int)) != cudaSuccess) return -1;
  if (v) {
    const int zero = 0;
    cudaMemcpyToSymbol(g_prompt_status, &zero, sizeof(int));
  }
  return v;
}

}  // namespace misa
