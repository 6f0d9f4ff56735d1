// Causal attention of packed prompts with grouped heads:
//   out_{i,h} = sum_{j <= i + o_b} softmax_j(scale q_{i,h} . k_{j,h'}) v_{j,h'},   o_b = keys - queries of b
// so the queries of a sequence are its last ones (o_b > 0 when earlier keys come from a cache), and a
// query with nothing to see (o_b < 0) gets zeros and a log-sum of minus infinity.
//
// What bounds it: 4 d operations for every (query, key, head) pair that is seen, on the tensor cores
// (4096 multiply-adds a clock and SM), and as much time again for the pair's exponential (16 a clock and
// SM): a 128 x 128 piece takes 2 x 512 clocks of products at d = 128 and 1024 of exponentials.  So a CTA
// works on two tiles of 128 queries at once: while one tile's scores go through the softmax, the tensor
// cores multiply for the other.  Measured, a pair of pieces takes 3250 clocks where the products alone
// would take 2048: Q K^T runs at 600 to 700 clocks for 512 (both operands come from shared memory, 128
// bytes a clock, all it has), and a tile's own chain (scores, weights, P V, the next Q K^T) is as long as
// that, because tensor memory has no room for a second set of scores.  4096 queries ending 32768 keys (16
// heads on 2): 840 us by itself, 1230 TFLOP/s, 0.74 of the measured bf16 rate; in a long run of calls, under the
// power cap, 953 us, 1080 TFLOP/s.
// Tried and slower: scores of 64 keys in two halves, two steps ahead (1139 us for 838); a quarter to half
// of the exponentials by a polynomial on the multiply-add units (860 to 927 for 858); reading the scores
// twice from tensor memory instead of holding them (1073 for 1055); outputs through TMA stores.
//
// Per CTA (one per SM): items of 256 queries of one head, tiles A and B, and the keys they see in ascending
// blocks of 128.  S = Q K^T and O += P V run on tcgen05 with fp32 accumulators in tensor memory
// (S_A, S_B, O_A, O_B: 128 columns each, all 512); P overwrites the first half of its S as bf16, the A
// operand of the second product.  Warp roles:
//   warps 0-3, 4-7  softmax of tile A, B: one thread a query row, so row maxima and sums need no
//                   exchange; also rescale O, normalise and write the output
//   warp 8          TMA producer: the two Q tiles, then K and V blocks through a ring of buffers
//   warp 9          MMA issuer (one elected thread) and owner of the tensor memory
//   warps 10, 11    guards: in the blocks where some query does not see every key they set to zero the
//                   value rows behind the sequence and every value that is not finite (a weight of
//                   zero times such a value would not be zero), before the product reads them
// The running maximum m is raised, and O rescaled, only when a row's scores pass it by 8 (base 2): O and
// the sum stay right for any m, and weights up to 2^8 lose nothing in bf16 or fp32.  Weights are rounded
// to bf16 (half a step, 2^-8 of the weight) for the product with V, of the same type; their sum is taken
// before, in fp32.  Values that are not finite and were set to zero are added to the rows that do see
// them at the end.
//
// Which CTA does what: with many long items one CTA takes one item, and the GPU's own dispatch evens them out;
// with short ones, or few long ones, 148 CTAs share the items' blocks equally, an item that a boundary cuts is
// left in pieces, and a last kernel joins them (130 queries over 20000 keys keep every SM busy).
// Every wait is bounded in time; a wait that runs out sets a device status word and all roles leave
// their loops, wait for their own copies and MMAs, and free tensor memory.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

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
// The compiler spills 356 bytes stored and 480 loaded a thread at d = 128 (252 and 368 at d = 64), much of it in
// the roles beside the softmax: 192 / 120 spills 248 and 320, 208 / 88 444 and 568.  200 / 104 is the one timed.
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
  static constexpr int kNumBars = 3 * kBufs + 2 * 7 + 1;
  static constexpr int kOffMisc = kOffBar + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kSmem = kOffMisc + 256 + 1024;      // + alignment slack
};

// Two consecutive tiles of queries of one sequence: rows [row, row + rows), which see keys of
// [key0, key0 + keys); query i of them sees keys j <= i + off.  count: blocks of keys they read, at least 1
// (an item that reads none still writes its outputs).
struct __align__(16) Pair {
  int row, rows, key0, keys;
  int off, count, pad0, pad1;
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

__device__ __forceinline__ Pair make_pair_of(int q0, int m, int k0, int l, int tile) {
  Pair p;
  p.row = q0 + tile * kPair;
  p.rows = min(kPair, m - tile * kPair);
  p.key0 = k0;
  p.keys = l;
  p.off = l - m + tile * kPair;
  p.count = max(1, max(p.blocks(0), p.blocks(1)));
  p.pad0 = p.pad1 = 0;
  return p;
}

// A place between blocks: block j of the item (pair, head).
struct __align__(16) Place {
  int pair, head, j, pad;
};

// Where an item is cut by the boundary in front of a CTA: the CTAs first .. last hold its pieces; pair < 0
// where nothing is cut, or the item's first cut lies further in front.
struct __align__(16) Cut {
  int pair, head, first, last;
};

// What a call of many or long items works from (prompt_plan_kernel): the pairs, and the sequence of items
// (pair by pair, the heads of a pair one after another) cut into pieces of equal cost, CTA c's from
// bounds[c] to bounds[c + 1].
struct Plan {
  Pair* pairs;     // null: CTA x takes item x, and no item is cut
  Place* bounds;   // [kCtas + 1]
  Cut* cuts;       // [kCtas]
  uint64_t* cost;  // [pairs] running costs of one head's items
  int most;        // room in `pairs`: what cu_q can hold where it does not decrease
  float* part;     // [2 kCtas][D][kPair] sums of a CTA's first (cut in front) and last (cut behind) item
  float* part_ml;  // [2 kCtas][2][kPair] their maxima and sums of weights
};

// An item costs its blocks and what its start and end take, in blocks.
constexpr int kItemCost = 4;
constexpr int kCtas = 148;
constexpr int64_t kManyItems = 4 * kCtas;

struct PromptArgs {
  const __nv_bfloat16* v;
  int64_t ldv;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int S, Tq, Tk, Hq, G;
  float c;                // scale times log2(e)
  __nv_bfloat16* out;
  float* lse;
  Plan plan;
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

// Warp-wide: lane l writes 8 consecutive columns of TMEM lane (taddr.lane + l).
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Warp-wide: lane l reads 16 consecutive columns of TMEM lane (taddr.lane + l); the values are there on return.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// 32 bytes, a whole sector, in one store; p is 32-byte aligned.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Warp-wide: lane l reads 8 consecutive columns of TMEM lane (taddr.lane + l); the values are there on return.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Keys and queries of sequence b, clamped to the tensors: q0, m, k0, l.
__device__ __forceinline__ int4 sequence(const PromptArgs& a, int b) {
  const int q0 = max(0, __ldg(a.cu_q + b)), q1 = min(a.Tq, __ldg(a.cu_q + b + 1));
  const int k0 = max(0, __ldg(a.cu_k + b)), k1 = min(a.Tk, __ldg(a.cu_k + b + 1));
  return make_int4(q0, max(0, q1 - q0), k0, max(0, k1 - k0));
}

// Without a plan: the pair of CTA x / Hq, pairs of every sequence from its last to its first.  False when
// there is none.  Every thread of the block calls it.
__device__ __forceinline__ bool find_pair(const PromptArgs& a, int pair, Pair& p, uint32_t* warp_tot, Pair* found,
                                          int* hit) {
  int base = 0;
  if (threadIdx.x == 0) *hit = 0;
  for (int b0 = 0; b0 < a.S; b0 += kThreads) {
    const int b = b0 + (int)threadIdx.x;
    const int4 q = b < a.S ? sequence(a, b) : make_int4(0, 0, 0, 0);
    const int tiles = (q.y + kPair - 1) / kPair;
    uint32_t total;
    const int before = base + (int)block_exclusive_scan((uint32_t)tiles, warp_tot, &total);
    if (pair >= before && pair < before + tiles) {
      *found = make_pair_of(q.x, q.y, q.z, q.w, tiles - 1 - (pair - before));
      *hit = 1;
    }
    __syncthreads();
    if (*hit) break;
    base += (int)total;
    if (base > pair) break;
  }
  if (a.S <= 0 || !*hit) return false;
  p = *found;
  return true;
}

constexpr int kPlanThreads = 512;
constexpr int kPlanShared = 2048;  // pairs whose running costs fit in shared memory

// The plan of one call, by one CTA.
__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const PromptArgs a) {
  __shared__ int base[kPlanThreads];
  __shared__ uint32_t warp_tot[32];
  __shared__ uint64_t run[kPlanShared];
  __shared__ Place bounds[kCtas + 1];
  __shared__ uint64_t carry;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n = 0;
  for (int b0 = 0; b0 < a.S; b0 += kPlanThreads) {
    const int b = b0 + (int)threadIdx.x;
    const int4 mine = b < a.S ? sequence(a, b) : make_int4(0, 0, 0, 0);
    uint32_t total;
    base[threadIdx.x] = n + (int)block_exclusive_scan((uint32_t)((mine.y + kPair - 1) / kPair), warp_tot, &total);
    __syncthreads();
    for (int x = warp; x < min(kPlanThreads, a.S - b0); x += kPlanThreads / 32) {
      const int4 q = sequence(a, b0 + x);
      const int tiles = (q.y + kPair - 1) / kPair;
      for (int t = lane; t < tiles && base[x] + t < a.plan.most; t += 32)
        a.plan.pairs[base[x] + t] = make_pair_of(q.x, q.y, q.z, q.w, t);
    }
    n = min(a.plan.most, n + (int)total);
    __syncthreads();
  }
  // running costs
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  for (int p0 = 0; p0 < n; p0 += kPlanThreads) {
    const int p = p0 + (int)threadIdx.x;
    uint32_t total;
    const uint32_t cost = p < n ? (uint32_t)(a.plan.pairs[p].count + kItemCost) : 0u;
    const uint32_t before = block_exclusive_scan(cost, warp_tot, &total);
    if (p < n) {
      const uint64_t v = carry + before;
      a.plan.cost[p] = v;
      if (p < kPlanShared) run[p] = v;
    }
    __syncthreads();
    if (threadIdx.x == 0) carry += total;
    __syncthreads();
  }
  const uint64_t W = carry * a.Hq, parts = W < kCtas ? W : kCtas, slack = W / (16 * kCtas);
  auto cost = [&](int p) { return p < kPlanShared ? run[p] : a.plan.cost[p]; };
  const int c = threadIdx.x;
  if (c <= kCtas) {
    Place at = {n, 0, 0, 0};
    const uint64_t x = c >= (int)parts ? W : W * c / parts;
    if (x < W) {
      int lo = 0, hi = n - 1;  // the last pair that starts at or before x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cost(mid) * a.Hq <= x) lo = mid;
        else hi = mid - 1;
      }
      const int blocks = a.plan.pairs[lo].count;
      const uint64_t each = (uint64_t)(blocks + kItemCost), in = x - cost(lo) * a.Hq;
      at.pair = lo;
      at.head = (int)(in / each);
      const uint64_t u = in - at.head * each;
      // an item is not cut for a sixteenth of a share, nor inside its fixed cost
      if (u <= kItemCost || u <= slack) {
        at.j = 0;
      } else if (each - u <= slack) {
        at.j = 0;
        if (++at.head == a.Hq) {
          at.head = 0;
          ++at.pair;
        }
      } else {
        at.j = (int)(u - kItemCost);
      }
    }
    bounds[c] = at;
    a.plan.bounds[c] = at;
  }
  __syncthreads();
  if (c < kCtas) {
    Cut cut = {-1, 0, 0, 0};
    const Place x = bounds[c];
    auto same = [&](const Place& y) { return y.pair == x.pair && y.head == x.head && y.j > 0; };
    if (c > 0 && x.j > 0 && !same(bounds[c - 1])) {
      int last = c;
      while (last + 1 < kCtas && same(bounds[last + 1])) ++last;
      cut = {x.pair, x.head, c - 1, last};
    }
    a.plan.cuts[c] = cut;
  }
}

// The work of one CTA, segment by segment: blocks [j0, j1) of the item (p, head).
struct Walk {
  Pair p;
  int head, j0, j1;
  int pair, end_pair, end_head, end_j;
  __device__ __forceinline__ void take() { j1 = pair == end_pair && head == end_head ? end_j : p.count; }
  // no segment left
  __device__ __forceinline__ bool over() const {
    return pair > end_pair || (pair == end_pair && (head > end_head || (head == end_head && j0 >= end_j)));
  }
  __device__ __forceinline__ void one(const Pair& q, int h) {
    p = q;
    head = h;
    j0 = 0;
    j1 = p.count;
    pair = 0;
    end_pair = 0;
    end_head = h;
    end_j = j1;
  }
  __device__ __forceinline__ bool begin(const PromptArgs& a, int cta) {
    const Place x = a.plan.bounds[cta], e = a.plan.bounds[cta + 1];
    pair = x.pair;
    head = x.head;
    j0 = x.j;
    end_pair = e.pair;
    end_head = e.head;
    end_j = e.j;
    if (over()) return false;
    p = a.plan.pairs[pair];
    take();
    return true;
  }
  __device__ __forceinline__ bool advance(const PromptArgs& a) {
    j0 = 0;  // a segment that others follow ends its item
    ++head;
    const bool next = head == a.Hq;
    if (next) {
      head = 0;
      ++pair;
    }
    if (over()) return false;
    if (next) p = a.plan.pairs[pair];
    take();
    return true;
  }
  // blocks of tile t in this segment
  __device__ __forceinline__ int from(int t) const { return min(j0, p.blocks(t)); }
  __device__ __forceinline__ int to(int t) const { return min(j1, p.blocks(t)); }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == p.count; }
  // whether block j has keys that some query of the pair does not see
  __device__ __forceinline__ bool guarded(int j) const {
    return (j < p.blocks(0) && p.masked(0, j)) || (j < p.blocks(1) && p.masked(1, j));
  }
};

// Adds to row i of a pair the values that are not finite and that it sees in blocks [from, to): the guards
// took them out of those that some query does not see whole.  v: the kv head's first value of the
// sequence; out (bf16, D in a row) or part (fp32, kPair apart): what this thread has just written.
template <int D>
__device__ __noinline__ void add_strange(const __nv_bfloat16* v, int64_t ldv, Pair p, int from, int to, int i,
                                         __nv_bfloat16* out, float* part) {
  const int end = min(p.keys, i + p.off + 1);
  for (int k = from * kRows; k < min(end, to * kRows); ++k) {
    const int j = k / kRows;
    if (!((j < p.blocks(0) && p.masked(0, j)) || (j < p.blocks(1) && p.masked(1, j)))) continue;
    for (int e = 0; e < D; ++e) {
      const float f = __bfloat162float(v[k * ldv + e]);
      if (isfinite(f)) continue;
      if (out) out[e] = __float2bfloat16_rn(__bfloat162float(out[e]) + f);
      else part[e * kPair] += f;
    }
  }
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
  // the last segment (plus one) in which a value that is not finite was set to zero, for every residue of its
  // number modulo 4.  It only grows, so that guards that are ahead of the softmax, by any number of segments,
  // cannot hide what they did in the softmax's own; what they did later costs it a search for nothing.
  int* odd = reinterpret_cast<int*>(misc + 4);
  Pair* found = reinterpret_cast<Pair*>(misc + 8);
  uint32_t* warp_tot = misc + 20;
  int* hit = reinterpret_cast<int*>(misc + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  Walk walk;
  if (a.plan.pairs == nullptr) {
    Pair p;
    if (!find_pair(a, blockIdx.x / a.Hq, p, warp_tot, found, hit)) return;
    walk.one(p, blockIdx.x % a.Hq);
  } else {
    pdl_wait();
    if (!walk.begin(a, blockIdx.x)) return;
  }

  const uint32_t bar0 = tc::smem_u32(sm + L::kOffBar);
  auto full = [&](int i) { return bar0 + 8 * i; };
  auto empty = [&](int i) { return bar0 + 8 * (NB + i); };
  auto vok = [&](int i) { return bar0 + 8 * (2 * NB + i); };
  auto qfull = [&](int t) { return bar0 + 8 * (3 * NB + t); };
  auto qempty = [&](int t) { return bar0 + 8 * (3 * NB + 2 + t); };
  auto sfull = [&](int t) { return bar0 + 8 * (3 * NB + 4 + t); };
  auto phalf = [&](int t) { return bar0 + 8 * (3 * NB + 6 + t); };
  auto pfull = [&](int t) { return bar0 + 8 * (3 * NB + 8 + t); };
  auto odone = [&](int t) { return bar0 + 8 * (3 * NB + 10 + t); };
  auto oread = [&](int t) { return bar0 + 8 * (3 * NB + 12 + t); };
  const uint32_t drain = bar0 + 8 * (3 * NB + 14);
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(qfull(t), 1);
      tc::mbar_init(qempty(t), 1);
      tc::mbar_init(sfull(t), 1);
      tc::mbar_init(phalf(t), 4);
      tc::mbar_init(pfull(t), 4);
      tc::mbar_init(odone(t), 1);
      tc::mbar_init(oread(t), 4);
    }
    for (int i = 0; i < NB; ++i) {
      tc::mbar_init(full(i), 1);
      tc::mbar_init(empty(i), 1);
      tc::mbar_init(vok(i), 2);
    }
    tc::mbar_init(drain, 1);
    *abort = 0;
    for (int x = 0; x < 4; ++x) odd[x] = 0;
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
  // every segment's blocks j0 .. j1 - 1 take turns in the ring, K before V

  if (warp < 8) {
    // ---------------- softmax ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2;
    const int i = t * kRows + (warp & 3) * 32 + lane;  // query of the pair
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * kRows, to = tmem + lanes + 2 * kRows + t * kRows;
    const float c = a.c;
    bool ok = true;
    uint32_t done = 0;  // blocks of this tile so far
    for (int seg = 0;; ++seg) {
      const int from = walk.from(t), to_ = walk.to(t);
      float m = -INFINITY, l = 0.f;  // maximum of the raw scores, sum of the weights
      for (int j = from; j < to_; ++j, ++done) {
        if (!wait_for(sfull(t), done & 1, abort)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int x = 0; x < 4; ++x) tc::tmem_ld32(ts + 32 * x, s[x]);
#pragma unroll
        for (int x = 0; x < 4; ++x) tc::tmem_ld_wait(s[x]);
        if (walk.p.masked(t, j)) {
          const int seen = min(walk.p.keys, i + walk.p.off + 1) - j * kRows;  // keys of this block that row i sees
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
          const uint32_t(&x)[32] = s[e / 16];
          const float2 y = make_float2(__uint_as_float(x[2 * (e % 16)]), __uint_as_float(x[2 * (e % 16) + 1]));
          const float2 z = __ffma2_rn(y, make_float2(c, c), make_float2(neg, neg));
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
            for (int x = 0; x < 4; ++x)
              top[x] = max3(top[x], __uint_as_float(s[x][2 * e]), __uint_as_float(s[x][2 * e + 1]));
          }
        }
        const float mx = max3(fmaxf(top[0], top[1]), top[2], top[3]);
        const bool raise = mx * c > m * c + kSlack;  // also the first score that is seen
        if (__any_sync(0xffffffffu, raise)) {
          if (j > from) {
            // O holds the blocks before this one once their product is through
            if (!wait_for(odone(t), (done - 1) & 1, abort)) {
              ok = false;
              break;
            }
            tc::tc_fence_after();
            const float f = raise && m != -INFINITY ? ex2((m - mx) * c) : 1.f;
            l *= f;
#pragma unroll 1
            for (int x = 0; x < D; x += 8) {
              uint32_t o[8];
              tmem_ld8(to + x, o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st8(to + x, o);
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
      if (ok && to_ > from && !wait_for(odone(t), (done - 1) & 1, abort)) ok = false;
      if (!ok) {
        give_up(abort);
        break;
      }
      tc::tc_fence_after();
      const Pair& p = walk.p;
      const bool whole = walk.whole();
      if (t * kRows + (warp & 3) * 32 < p.rows || to_ > from) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int slot = 2 * blockIdx.x + (walk.j0 == 0 ? 1 : 0);
        __nv_bfloat16* out = a.out + ((int64_t)(p.row + i) * a.Hq + walk.head) * D;
        float* part = a.plan.part + (int64_t)slot * D * kPair + i;
        // a row's outputs go out by whole sectors of 32 bytes (packed prompts of 200 to 4096 tokens: 473 us, 491 by
        // halves of them)
        const bool sectors = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
        // sixteen outputs at a time, in a loop of few instructions: once an item, this code is not in the
        // instruction cache when it runs
#pragma unroll 1
        for (int x = 0; x < D; x += 16) {
          uint32_t o[16];
          if (to_ > from) {
            tmem_ld16(to + x, o);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0u;
          }
          if (!whole) {
#pragma unroll
            for (int e = 0; e < 16; ++e) part[(x + e) * kPair] = __uint_as_float(o[e]);
          } else {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __nv_bfloat162 h =
                  __floats2bfloat162_rn(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
              w[e] = *reinterpret_cast<const uint32_t*>(&h);
            }
            if (i < p.rows) {
              if (sectors) {
                store32(out + x, w);
              } else {
                reinterpret_cast<uint4*>(out + x)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(out + x)[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          }
        }
        if (to_ > from) {  // the next segment may overwrite O
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_relaxed(oread(t));
        }
        if (!whole) {
          a.plan.part_ml[(slot * 2) * kPair + i] = m;
          a.plan.part_ml[(slot * 2 + 1) * kPair + i] = l;
        } else if (a.lse && i < p.rows) {
          a.lse[((int64_t)p.row + i) * a.Hq + walk.head] =
              l == 0.f ? -INFINITY : m * c * 0.693147180559945309f + logf(l);
        }
        if (*reinterpret_cast<volatile int*>(odd + (seg & 3)) > seg && i < p.rows)
          add_strange<D>(a.v + (int64_t)p.key0 * a.ldv + (walk.head / a.G) * D, a.ldv, p, from, to_, i,
                         whole ? out : nullptr, part);
      }
      if (!walk.advance(a)) break;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kLoadWarp) {
      // ---------------- TMA producer ----------------
      if (elect_one()) {
        bool ok = true;
        uint32_t u = 0, q[2] = {0, 0};  // ring buffers and Q tiles filled so far
        auto wait = [&](uint32_t bar, uint32_t parity) {
          if (ok && !wait_for(bar, parity, abort)) ok = false;
          return ok;
        };
        do {
          const Pair& p = walk.p;
          const int hk = walk.head / a.G;
          const bool has[2] = {walk.to(0) > walk.from(0), walk.to(1) > walk.from(1)};
          auto q_tile = [&](int t) {
            if (q[t] > 0 && !wait(qempty(t), (q[t] - 1) & 1)) return;
            ++q[t];
            tc::mbar_arrive_expect_tx(qfull(t), L::kTileBytes);
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
              tc::tma_load_2d(qbase + t * L::kTileBytes + x * L::kHalfBytes, &qmap, walk.head * D + x * 64,
                              p.row + t * kRows, qfull(t));
          };
          const int j1 = max(walk.to(0), walk.to(1));
          if (has[0]) q_tile(0);
          for (int j = walk.j0; ok && j < j1; ++j) {
            for (int side = 0; ok && side < 2; ++side, ++u) {
              const int b = u % NB;
              if (u >= NB && !wait(empty(b), ((u / NB) - 1) & 1)) break;
              tc::mbar_arrive_expect_tx(full(b), L::kTileBytes);
#pragma unroll
              for (int x = 0; x < D / 64; ++x)
                tc::tma_load_2d(ring + b * L::kTileBytes + x * L::kHalfBytes, side ? &vmap : &kmap, hk * D + x * 64,
                                p.key0 + j * kRows, full(b));
              if (j == walk.j0 && side == 0 && has[1]) q_tile(1);
            }
          }
        } while (ok && walk.advance(a));
        if (!ok) give_up(abort);
        // every issued copy lands before the CTA exits
        for (int t = 0; t < 2; ++t)
          if (q[t] > 0) wait_for(qfull(t), (q[t] - 1) & 1, nullptr);
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
        // One segment's blocks of either tile, [f0, t0) and [f1, t1), and the ring turn of its block j0
        struct Seg {
          int f0, t0, f1, t1, j0, j1;
          uint32_t turn;
          __device__ __forceinline__ int from(int t) const { return t ? f1 : f0; }
          __device__ __forceinline__ int to(int t) const { return t ? t1 : t0; }
          // the last tile that reads block j
          __device__ __forceinline__ bool last(int t, int j) const { return t == 1 || j < f1 || j >= t1; }
        };
        auto segment = [&](uint32_t turn) {
          Seg g;
          g.f0 = walk.from(0);
          g.t0 = walk.to(0);
          g.f1 = walk.from(1);
          g.t1 = walk.to(1);
          g.j0 = walk.j0;
          g.j1 = max(g.t0, g.t1);
          g.turn = turn;
          return g;
        };
        uint32_t qn0 = 0, qn1 = 0, on0 = 0, on1 = 0, dn0 = 0, dn1 = 0;  // Q tiles, outputs and blocks begun, by tile
        auto scores = [&](const Seg& g, const int t, int j) {  // S_t = Q_t K_j^T
          const uint32_t u = g.turn + 2 * (j - g.j0), b = u % NB;
          if (j == g.from(t)) {
            uint32_t& qn = t ? qn1 : qn0;
            if (!wait(qfull(t), qn & 1)) return;
            ++qn;
          }
          if (!wait(full(b), (u / NB) & 1)) return;
          const uint64_t qd = tc::sw128_kmajor_desc(qbase + t * L::kTileBytes);
          const uint64_t kd = tc::sw128_kmajor_desc(ring + b * L::kTileBytes);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t at = ((kk / 4) * L::kHalfBytes + (kk % 4) * 32) >> 4;
            tc::mma_bf16(tmem + t * kRows, qd + at, kd + at, idesc_s, kk != 0);
          }
          tc::mma_commit(sfull(t));
          if (j + 1 == g.to(t)) tc::mma_commit(qempty(t));
          if (g.last(t, j)) tc::mma_commit(empty(b));
        };
        auto values = [&](const Seg& g, const int t, int j) {  // O_t += P_t V_j
          const uint32_t u = g.turn + 2 * (j - g.j0) + 1, b = u % NB;
          uint32_t& dn = t ? dn1 : dn0;
          if (!wait(vok(b), (u / NB) & 1)) return;
          if (j == g.from(t)) {
            uint32_t& on = t ? on1 : on0;
            if (on > 0 && !wait(oread(t), (on - 1) & 1)) return;
            ++on;
          }
          const uint64_t vd = sw128_mnmajor_desc(ring + b * L::kTileBytes, L::kHalfBytes);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!wait(half ? pfull(t) : phalf(t), dn & 1)) return;
            tc::tc_fence_after();  // after the weights' stores to tensor memory, by other threads
#pragma unroll
            for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
              mma_bf16_ts(tmem + 2 * kRows + t * kRows, tmem + t * kRows + kk * 8, vd + kk * (2048 >> 4), idesc_o,
                          (j > g.from(t)) || kk != 0);
          }
          tc::mma_commit(odone(t));
          if (g.last(t, j)) tc::mma_commit(empty(b));
          ++dn;
        };
        Seg g = segment(0);
        if (g.t0 > g.f0) scores(g, 0, g.f0);
        if (ok && g.t1 > g.f1) scores(g, 1, g.f1);
        while (ok) {
          const bool more = walk.advance(a);
          Seg next = g;
          if (more) next = segment(g.turn + 2 * (uint32_t)max(0, g.j1 - g.j0));
          // a tile's first scores of the next segment follow its last block of this one, unless the other tile
          // has more than one block to go: the ring could not hold what lies between
          bool begun0 = false, begun1 = false;
          for (int j = g.j0; ok && j < g.j1; ++j) {
            const bool ahead = more && j + 2 >= g.j1;
            if (j >= g.f0 && j < g.t0) {
              values(g, 0, j);
              if (ok && j + 1 < g.t0) {
                scores(g, 0, j + 1);
              } else if (ok && ahead && next.t0 > next.f0) {
                scores(next, 0, next.f0);
                begun0 = true;
              }
            }
            if (ok && j >= g.f1 && j < g.t1) {
              values(g, 1, j);
              if (ok && j + 1 < g.t1) {
                scores(g, 1, j + 1);
              } else if (ok && ahead && j + 1 == g.j1 && next.t1 > next.f1 && (begun0 || next.t0 <= next.f0)) {
                // (behind the first tile's: the second one's use of a block is taken to be the last)
                scores(next, 1, next.f1);
                begun1 = true;
              }
            }
          }
          if (!ok || !more) break;
          g = next;
          if (!begun0 && g.t0 > g.f0) scores(g, 0, g.f0);
          if (ok && !begun1 && g.t1 > g.f1) scores(g, 1, g.f1);
        }
        if (!ok) give_up(abort);
        // every issued MMA completes before tensor memory is freed
        tc::mma_commit(drain);
        wait_for(drain, 0, nullptr);
      }
    } else {
      // ---------------- guards ----------------
      bool ok = true;
      uint32_t u = 1;  // ring turn of the next V
      for (int seg = 0;; ++seg) {
        for (int j = walk.j0; ok && j < max(walk.to(0), walk.to(1)); ++j, u += 2) {
          const uint32_t b = u % NB;
          if (!wait_for(full(b), (u / NB) & 1, abort)) {
            ok = false;
            break;
          }
          // passed on all the same: a guard that fell behind by a turn of the ring would miss its phase
          if (!walk.guarded(j)) {
            if (lane == 0) tc::mbar_arrive(vok(b));
            continue;
          }
          const int there = walk.p.keys - j * kRows;  // rows from here on belong to no key of the sequence
          const int first = (warp - kGuardWarp) * (kRows / 2);
          uint8_t* v = sm + L::kOffRing + b * L::kTileBytes;
          // a 16-bit number whose exponent is all ones carries into its top bit
          auto hit = [](uint32_t z) { return ((z & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
          auto clean = [&](uint32_t z) { return z & ~((hit(z) >> 15) * 0xffffu); };
          constexpr int kPieces = (kRows / 2) * (D / 8);  // of 16 bytes, 8 a row and box of 64 dims
          auto piece = [&](int x) {
            const int half = x / (kRows / 2 * 8), y = x % (kRows / 2 * 8);
            return reinterpret_cast<uint4*>(v + half * L::kHalfBytes + (first + y / 8) * 128 + (y % 8) * 16);
          };
          bool changed = false, bad = false;
          if (first + kRows / 2 > there) {
            for (int x = lane; x < kPieces; x += 32)
              if (first + x % (kRows / 2 * 8) / 8 >= there) *piece(x) = make_uint4(0u, 0u, 0u, 0u);
            changed = true;
          }
#pragma unroll 1
          for (int x0 = lane; x0 < kPieces; x0 += 32 * 8) {
            uint4 w[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) w[y] = *piece(x0 + 32 * y);
            uint32_t any = 0;
#pragma unroll
            for (int y = 0; y < 8; ++y) any |= hit(w[y].x) | hit(w[y].y) | hit(w[y].z) | hit(w[y].w);
            if (any) {
#pragma unroll 1
              for (int y = 0; y < 8; ++y) {
                uint4* p = piece(x0 + 32 * y);
                const uint4 z = *p;
                *p = make_uint4(clean(z.x), clean(z.y), clean(z.z), clean(z.w));
              }
              changed = bad = true;
            }
          }
          if (bad) atomicMax(odd + (seg & 3), seg + 1);
          if (changed) tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(vok(b));
        }
        if (!ok || !walk.advance(a)) break;
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

// Joins the pieces of the items that a boundary between CTAs cuts: CTA (c, y) takes 16 output columns of
// the item whose first cut lies in front of CTA c + 1, one thread a row.
template <int D>
__global__ void __launch_bounds__(kPair) prompt_join_kernel(const PromptArgs a) {
  pdl_wait();
  const Cut cut = a.plan.cuts[blockIdx.x + 1];
  if (cut.pair < 0) return;
  const Pair p = a.plan.pairs[cut.pair];
  const int i = threadIdx.x, d0 = blockIdx.y * 16;
  if (i >= p.rows) return;
  // the first piece is its CTA's last, the others their CTAs' first
  auto slot = [&](int c) { return 2 * c + (c == cut.first ? 1 : 0); };
  float top = -INFINITY;
  for (int c = cut.first; c <= cut.last; ++c) top = fmaxf(top, a.plan.part_ml[(slot(c) * 2) * kPair + i]);
  float sum = 0.f, o[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] = 0.f;
  for (int c = cut.first; c <= cut.last; ++c) {
    const int s = slot(c);
    const float l = a.plan.part_ml[(s * 2 + 1) * kPair + i];
    if (l == 0.f) continue;  // saw nothing
    const float f = ex2((a.plan.part_ml[(s * 2) * kPair + i] - top) * a.c);
    sum += f * l;
    const float* src = a.plan.part + ((int64_t)s * D + d0) * kPair + i;
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] += f * src[e * kPair];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * e] * inv, o[2 * e + 1] * inv);
    w[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  uint4* dst = reinterpret_cast<uint4*>(a.out + ((int64_t)(p.row + i) * a.Hq + cut.head) * D + d0);
  dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (a.lse && blockIdx.y == 0)
    a.lse[((int64_t)p.row + i) * a.Hq + cut.head] =
        sum == 0.f ? -INFINITY : top * a.c * 0.693147180559945309f + logf(sum);
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

int64_t most_pairs(int S, int Tq) { return (int64_t)Tq / kPair + std::min(S, Tq); }

// Whether a call goes without a plan, one item a CTA: where the items are few enough for one CTA an SM and
// none is long (32 blocks of keys at most), so that cutting them up would not pay for the two launches it
// adds, and where they are many and take long enough (more than 8 blocks of keys a sequence) for the GPU's own
// dispatch to even them out.  (Short ones gain from CTAs that stay: their loads and first scores go ahead of
// the last item's end.  32 heads, sequences of 256 tokens: 218 us for 317; of 1024: 407 for 417; of 2048: 549
// for 540; of 4096: 867 for 820.)
bool plain_call(int S, int Tq, int Tk, int Hq) {
  const int64_t items = most_pairs(S, Tq) * Hq;
  return (items > kManyItems && Tk > 8 * kRows * (int64_t)S) || (items <= kCtas && Tk <= 32 * kRows);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <int D>
bool launch_d(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const PromptArgs& a,
              cudaStream_t s) {
  static_assert(Lay<D>::kSmem <= 232448, "shared memory of the prompt kernel exceeds 227 KB");
  if (cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kSmem) != cudaSuccess)
    return false;
  if (a.plan.pairs == nullptr) {
    prompt_kernel<D><<<(unsigned)(most_pairs(a.S, a.Tq) * a.Hq), kThreads, Lay<D>::kSmem, s>>>(qm, km, vm, a);
    return true;
  }
  prompt_plan_kernel<<<1, kPlanThreads, 0, s>>>(a);
  launch_pdl(prompt_kernel<D>, dim3(kCtas), dim3(kThreads), Lay<D>::kSmem, s, qm, km, vm, a);
  launch_pdl(prompt_join_kernel<D>, dim3(kCtas - 1, D / 16), dim3(kPair), 0, s, a);
  return true;
}

}  // namespace

size_t prompt_ws_bytes(int S, int Tq, int Tk, int Hq, int d) {
  if (S <= 0 || Tq <= 0 || plain_call(S, Tq, Tk, Hq)) return 0;
  return up256(sizeof(Pair) * most_pairs(S, Tq)) + up256(sizeof(Place) * (kCtas + 1)) + up256(sizeof(Cut) * kCtas) +
         up256(sizeof(uint64_t) * most_pairs(S, Tq)) +
         up256(sizeof(float) * 2 * kCtas * (size_t)kPair * d) + up256(sizeof(float) * 4 * kCtas * kPair);
}

bool launch_prompt_attention(const void* q, const void* k, const void* v, int64_t ldq, int64_t ldk, int64_t ldv,
                             const int32_t* cu_q, const int32_t* cu_k, int S, int Tq, int Tk, int Hq, int Hkv, int d,
                             float scale, void* out, float* lse, void* ws, cudaStream_t s) {
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
  a.plan = {};
  if (!plain_call(S, Tq, Tk, Hq)) {
    char* p = static_cast<char*>(ws);
    a.plan.pairs = reinterpret_cast<Pair*>(p);
    p += up256(sizeof(Pair) * most_pairs(S, Tq));
    a.plan.bounds = reinterpret_cast<Place*>(p);
    p += up256(sizeof(Place) * (kCtas + 1));
    a.plan.cuts = reinterpret_cast<Cut*>(p);
    p += up256(sizeof(Cut) * kCtas);
    a.plan.cost = reinterpret_cast<uint64_t*>(p);
    p += up256(sizeof(uint64_t) * most_pairs(S, Tq));
    a.plan.most = (int)most_pairs(S, Tq);
    a.plan.part = reinterpret_cast<float*>(p);
    p += up256(sizeof(float) * 2 * kCtas * (size_t)kPair * d);
    a.plan.part_ml = reinterpret_cast<float*>(p);
  }
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
