// Which tokens of a cache stay when it is thinned to `keep` of them by the attention weight they have
// gathered: the first `sink`, the last `recent`, and of those between the ones with the largest summed
// weight (ties to the lower token).  One CTA per sequence: three passes over the row's order keys (11,
// 11 and 10 bits) find the last kept key and how many of its equals stay, a fourth writes the kept
// tokens in order, each at the number of kept tokens before it.
#include "kernels.cuh"

namespace misa {

namespace {

constexpr int kEvictThreads = 1024;
constexpr int kEvictBins = 2048;

// Order of the summed weights; NaN counts as the smallest.
__device__ __forceinline__ uint32_t weight_key(float f) { return f == f ? order_key(f) : 0u; }

__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const float* __restrict__ acc, int64_t ld,
                                                                     const int32_t* __restrict__ n, int L, int keep,
                                                                     int sink, int recent, int32_t* __restrict__ idx,
                                                                     int32_t* __restrict__ n_out,
                                                                     float* __restrict__ acc_out, int64_t ld_out) {
  __shared__ uint32_t hist[kEvictBins];
  __shared__ uint32_t warp_tot[32];
  __shared__ uint32_t found[2];
  const int t = blockIdx.x;
  const float* row = acc + (int64_t)t * ld;
  const int nt = clamp_len(n[t], L);
  const int kept = min(nt, keep);
  int32_t* out = idx + (int64_t)t * keep;
  float* aout = acc_out ? acc_out + (int64_t)t * ld_out : nullptr;
  if (threadIdx.x == 0) n_out[t] = kept;
  for (int j = kept + threadIdx.x; j < keep; j += kEvictThreads) out[j] = -1;
  if (aout)
    for (int64_t j = kept + threadIdx.x; j < ld_out; j += kEvictThreads) aout[j] = 0.f;
  const int s0 = min(sink, nt), s1 = nt - min(recent, nt);
  uint32_t want = nt > keep ? (uint32_t)(keep - sink - recent) : 0u;  // kept of [s0, s1)
  uint32_t cut = 0u;  // the smallest kept key, of which `want` stay in the end
  if (nt > keep && want > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = threadIdx.x; i < kEvictBins; i += kEvictThreads) hist[i] = 0;
      __syncthreads();
      for (int s = s0 + threadIdx.x; s < s1; s += kEvictThreads) {
        const uint32_t k = weight_key(__ldg(row + s));
        if (pass == 0 || (k >> (shift + bits)) == (cut >> (shift + bits)))
          atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
      }
      __syncthreads();
      // thread i owns bins [top - 2 i - 1, top - 2 i], from the largest down
      const int b = kEvictBins - 1 - 2 * (int)threadIdx.x;
      const uint32_t h0 = hist[b], h1 = hist[b - 1];
      uint32_t total;
      const uint32_t before = block_exclusive_scan(h0 + h1, warp_tot, &total);
      if (before < want && want <= before + h0) {
        found[0] = b;
        found[1] = want - before;
      } else if (before + h0 < want && want <= before + h0 + h1) {
        found[0] = b - 1;
        found[1] = want - before - h0;
      }
      __syncthreads();
      cut |= found[0] << shift;
      want = found[1];
      __syncthreads();
    }
  }
  // kept tokens in order
  uint32_t base = 0, tie = 0;
  for (int c0 = 0; c0 < nt; c0 += kEvictThreads) {
    const int s = c0 + threadIdx.x;
    const float a = s < nt ? __ldg(row + s) : 0.f;
    const uint32_t k = weight_key(a);
    const bool held = s < nt && (nt <= keep || s < s0 || s >= s1);
    const bool mid = s < nt && !held && want > 0;
    const bool eq = mid && k == cut;
    uint32_t ties, all;
    const uint32_t eb = block_exclusive_scan(eq ? 1u : 0u, warp_tot, &ties);
    const bool stay = held || (mid && k > cut) || (eq && tie + eb < want);
    const uint32_t at = base + block_exclusive_scan(stay ? 1u : 0u, warp_tot, &all);
    if (stay) {
      out[at] = s;
      if (aout) aout[at] = a;
    }
    base += all;
    tie += ties;
  }
}

}  // namespace

void launch_evict_select(const float* acc, int64_t ld, const int32_t* n, int T, int L, int keep, int sink, int recent,
                         int32_t* idx, int32_t* n_out, float* acc_out, int64_t ld_out, cudaStream_t s) {
  if (T <= 0) return;
  evict_select_kernel<<<T, kEvictThreads, 0, s>>>(acc, ld, n, L, keep, sink, recent, idx, n_out, acc_out, ld_out);
}

}  // namespace misa
