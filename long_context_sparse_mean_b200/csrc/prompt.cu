// Causal attention of packed prompts with grouped heads:
//   out_{i,h} = sum_{j <= i + o_b} softmax_j(scale q_{i,h} . k_{j,h'}) v_{j,h'},   o_b = keys - queries of b
// so the queries of a sequence are its last ones (o_b > 0 when earlier keys come from a cache), and a
// query with nothing to see (o_b < 0) gets zeros and a log-sum of minus infinity.
#include "kernels.cuh"

namespace misa {

namespace {

// One warp per (query row, head): lanes hold d / 32 dimensions each.
template <int D>
__global__ void __launch_bounds__(256) prompt_rows_kernel(const __nv_bfloat16* __restrict__ q,
                                                          const __nv_bfloat16* __restrict__ k,
                                                          const __nv_bfloat16* __restrict__ v, int64_t ldq, int64_t ldk,
                                                          int64_t ldv, const int32_t* __restrict__ cu_q,
                                                          const int32_t* __restrict__ cu_k, int S, int Tq, int Tk, int Hq,
                                                          int G, float scale, __nv_bfloat16* __restrict__ out,
                                                          float* __restrict__ lse) {
  constexpr int E = D / 32;
  const int64_t id = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (id >= (int64_t)Tq * Hq) return;
  const int row = (int)(id / Hq), h = (int)(id % Hq);
  if (row < __ldg(cu_q) || row >= __ldg(cu_q + S)) return;
  int lo = 0, hi = S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu_q + mid) <= row) lo = mid;
    else hi = mid;
  }
  const int k0 = max(0, __ldg(cu_k + lo)), k1 = min(Tk, __ldg(cu_k + lo + 1));
  const int seen = min(k1 - k0, row - __ldg(cu_q + lo) + 1 + (k1 - k0) - (__ldg(cu_q + lo + 1) - __ldg(cu_q + lo)));
  float qf[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qf[e] = __bfloat162float(q[(int64_t)row * ldq + h * D + lane * E + e]) * scale * 1.44269504088896341f;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < seen; ++j) {
    const int64_t at = (int64_t)(k0 + j), hk = (h / G) * D + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += qf[e] * __bfloat162float(k[at * ldk + hk + e]);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float next = fmaxf(m, s), f = exp2f(m - next), p = exp2f(s - next);
    m = next;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * __bfloat162float(v[at * ldv + hk + e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    out[((int64_t)row * Hq + h) * D + lane * E + e] = __float2bfloat16_rn(seen > 0 ? o[e] / l : 0.f);
  if (lse && lane == 0) lse[(int64_t)row * Hq + h] = seen > 0 ? (m + log2f(l)) * 0.693147180559945309f : -INFINITY;
}

}  // namespace

void launch_prompt_attention(const void* q, const void* k, const void* v, int64_t ldq, int64_t ldk, int64_t ldv,
                             const int32_t* cu_q, const int32_t* cu_k, int S, int Tq, int Tk, int Hq, int Hkv, int d,
                             float scale, void* out, float* lse, cudaStream_t s) {
  if (S <= 0 || Tq <= 0) return;
  const unsigned grid = (unsigned)(((int64_t)Tq * Hq + 7) / 8);
  const auto* qb = static_cast<const __nv_bfloat16*>(q);
  const auto* kb = static_cast<const __nv_bfloat16*>(k);
  const auto* vb = static_cast<const __nv_bfloat16*>(v);
  auto* ob = static_cast<__nv_bfloat16*>(out);
  if (d == 128)
    prompt_rows_kernel<128><<<grid, 256, 0, s>>>(qb, kb, vb, ldq, ldk, ldv, cu_q, cu_k, S, Tq, Tk, Hq, Hq / Hkv, scale, ob, lse);
  else
    prompt_rows_kernel<64><<<grid, 256, 0, s>>>(qb, kb, vb, ldq, ldk, ldv, cu_q, cu_k, S, Tq, Tk, Hq, Hq / Hkv, scale, ob, lse);
}

}  // namespace misa
