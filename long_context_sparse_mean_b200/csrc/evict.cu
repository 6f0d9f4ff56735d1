// Which tokens of a cache stay when it is thinned to `keep` of them by the attention weight they have
// gathered: the first `sink`, the last `recent`, and of those between the ones with the largest summed
// weight (ties to the lower token).
//
// Little is read and written, so a call lasts as long as its chain of dependent steps; the work of a row is
// spread over a cluster of 8 CTAs to keep each step short, and its weights stay in registers, a run of
// consecutive tokens a thread, where the runs are short enough.  Three histogram passes over the order keys
// (11, 11 and 10 bits) find the last kept key and how many of its equals stay: each CTA counts its tokens in
// shared memory, and all add up the eight histograms through distributed shared memory.  Then every thread
// counts the kept tokens of its run, one scan over the CTA and the counts of the CTAs before it say where they
// go, and they are written in order.
// n_out may be n: every thread of a row's CTAs reads its length before a barrier, the new one is written behind it.
// 16 rows of up to 32768 tokens: 19.6 us (one CTA a row, with a scan for every 1024 tokens: 55.7; read in every
// pass: 22); one row of 1000 tokens: 8.3 us a replay.
#include <cooperative_groups.h>

#include "kernels.cuh"

namespace cg = cooperative_groups;

namespace misa {

namespace {

constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kOneCta = 4096;  // rows up to here take one CTA: a cluster's barriers cost more than they save
static_assert(kBins == 4 * kThreads, "a thread owns four bins");

// Order of the summed weights; NaN counts as the smallest.
__device__ __forceinline__ uint32_t weight_key(float f) { return f == f ? order_key(f) : 0u; }

template <int kCluster, int HOLD>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    evict_select_kernel(const float* __restrict__ acc, int64_t ld, const int32_t* n, int L, int keep, int sink,
                        int recent, int32_t* __restrict__ idx, int32_t* n_out, float* __restrict__ acc_out,
                        int64_t ld_out) {
  __shared__ __align__(16) uint32_t hist[3][kBins];
  __shared__ uint32_t warp_tot[32];
  __shared__ uint32_t found[2];
  __shared__ uint32_t counts[2];  // of this CTA's tokens: kept for sure, equal to the cut
  cg::cluster_group cluster = cg::this_cluster();
  const int t = blockIdx.x / kCluster, rank = (int)cluster.block_rank();
  const float* row = acc + (int64_t)t * ld;
  const int nt = clamp_len(n[t], L);
  const int kept = min(nt, keep);
  int32_t* out = idx + (int64_t)t * keep;
  float* aout = acc_out ? acc_out + (int64_t)t * ld_out : nullptr;
  const int me = rank * kThreads + (int)threadIdx.x;
  for (int j = kept + me; j < keep; j += kCluster * kThreads) out[j] = -1;
  if (aout)
    for (int64_t j = kept + me; j < ld_out; j += kCluster * kThreads) aout[j] = 0.f;
  if (nt <= keep) {  // the whole cluster alike
    if (kCluster > 1) cluster.sync();
    else __syncthreads();
    if (rank == 0 && threadIdx.x == 0) n_out[t] = kept;
    for (int s = me; s < nt; s += kCluster * kThreads) {
      out[s] = s;
      if (aout) aout[s] = __ldg(row + s);
    }
    return;
  }
  const int s0 = sink, s1 = nt - recent;          // the tokens that compete
  uint32_t want = (uint32_t)(keep - sink - recent);  // how many of them stay
  uint32_t cut = 0u;                               // the smallest kept key, of which `want` stay in the end
  const bool choose = want > 0;
  // runs of consecutive tokens, one a thread; their keys stay in registers where a run is at most HOLD
  const int run = (nt + kCluster * kThreads - 1) / (kCluster * kThreads);
  const int r0 = (int)min((int64_t)nt, (int64_t)me * run), r1 = min(nt, r0 + run);
  float held_w[HOLD > 0 ? HOLD : 1];
#pragma unroll
  for (int i = 0; i < HOLD; ++i) held_w[i] = r0 + i < r1 ? __ldg(row + r0 + i) : 0.f;
  auto each = [&](auto f) {  // of the thread's tokens, in order
    if (HOLD > 0) {
#pragma unroll
      for (int i = 0; i < HOLD; ++i)
        if (r0 + i < r1) f(r0 + i, held_w[i]);
    } else {
#pragma unroll 4
      for (int s = r0; s < r1; ++s) f(s, __ldg(row + s));
    }
  };
  auto held = [&](int s) { return s < s0 || s >= s1; };
  if (choose) {
    for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) hist[0][i] = 0;
    __syncthreads();
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      auto count = [&](int s, float w) {
        const uint32_t k = weight_key(w);
        if (!held(s) && (pass == 0 || (k >> (shift + bits)) == (cut >> (shift + bits))))
          atomicAdd(&hist[pass][(k >> shift) & ((1u << bits) - 1)], 1u);
      };
      if (HOLD > 0) {
        each(count);
      } else {  // in any order: neighbours by neighbouring threads
#pragma unroll 8
        for (int s = s0 + me; s < s1; s += kCluster * kThreads) count(s, __ldg(row + s));
      }
      if (kCluster > 1) cluster.sync();
      else __syncthreads();
      // thread i owns four bins, the largest first
      const int b0 = kBins - 4 * ((int)threadIdx.x + 1);
      uint32_t h[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int x = 0; x < kCluster; ++x) {
        const uint32_t* p = kCluster > 1 ? cluster.map_shared_rank(&hist[pass][b0], x) : &hist[pass][b0];
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        h[3] += v.x;
        h[2] += v.y;
        h[1] += v.z;
        h[0] += v.w;
      }
      uint32_t total;
      uint32_t before = block_exclusive_scan(h[0] + h[1] + h[2] + h[3], warp_tot, &total);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (before < want && want <= before + h[x]) {
          found[0] = (uint32_t)(b0 + 3 - x);
          found[1] = want - before;
        }
        before += h[x];
      }
      __syncthreads();
      cut |= found[0] << shift;
      want = found[1];
      __syncthreads();
    }
  }
  uint32_t sure = 0, equal = 0;
  each([&](int s, float w) {
    const uint32_t k = weight_key(w);
    sure += held(s) || (choose && k > cut);
    equal += !held(s) && choose && k == cut;
  });
  uint32_t sure_all, equal_all;
  uint32_t sure_at = block_exclusive_scan(sure, warp_tot, &sure_all);
  uint32_t equal_at = block_exclusive_scan(equal, warp_tot, &equal_all);
  if (threadIdx.x == 0) {
    counts[0] = sure_all;
    counts[1] = equal_all;
  }
  if (kCluster > 1) cluster.sync();
  for (int x = 0; x < rank; ++x) {
    const uint32_t* c = cluster.map_shared_rank(counts, x);
    sure_at += c[0];
    equal_at += c[1];
  }
  each([&](int s, float v) {
    const uint32_t k = weight_key(v);
    const bool eq = !held(s) && choose && k == cut;
    const bool stay = held(s) || (choose && k > cut) || (eq && equal_at < want);
    if (stay) {
      // kept before it: those that stay for sure, and the first equals up to `want`
      const uint32_t at = sure_at + min(equal_at, want);
      out[at] = s;
      if (aout) aout[at] = v;
    }
    sure_at += stay && !eq;
    equal_at += eq;
  });
  if (kCluster > 1) cluster.sync();  // no CTA leaves while another may read its counts
  if (rank == 0 && threadIdx.x == 0) n_out[t] = kept;
}

}  // namespace

void launch_evict_select(const float* acc, int64_t ld, const int32_t* n, int T, int L, int keep, int sink, int recent,
                         int32_t* idx, int32_t* n_out, float* acc_out, int64_t ld_out, cudaStream_t s) {
  if (T <= 0) return;
  auto run = [&](auto kernel, int cluster) {
    kernel<<<T * cluster, kThreads, 0, s>>>(acc, ld, n, L, keep, sink, recent, idx, n_out, acc_out, ld_out);
  };
  if (L <= kOneCta) run(evict_select_kernel<1, kOneCta / kThreads>, 1);
  // registers for as long a run as the longest row has, up to 32 (one row of 128K tokens with both compactions:
  // 115 us, 129 us when it is read in every pass)
  else if (L <= 8 * 8 * kThreads) run(evict_select_kernel<8, 8>, 8);
  else if (L <= 8 * 16 * kThreads) run(evict_select_kernel<8, 16>, 8);
  else if (L <= 8 * 32 * kThreads) run(evict_select_kernel<8, 32>, 8);
  else run(evict_select_kernel<8, 0>, 8);
}

}  // namespace misa
