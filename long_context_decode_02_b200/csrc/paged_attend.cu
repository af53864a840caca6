// Attention over the paged 8-bit cache for the last n_q tokens of every sequence:
//   z_t = (q . k_code_t) k_scale / sqrt(d),  out = sum_t softmax(z)_t v_code_t v_scale.
// One CTA per (query, query head, sequence); a warp takes every fourth token, a lane d/32
// elements of it, with an online softmax in fp32; the warps merge in shared memory.
#include "paged_common.cuh"

namespace lowram {
namespace {

constexpr int kWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) paged_attend_kernel(const PagedArgs a) {
  constexpr int E = D / 32;
  const int j = blockIdx.x, hq = blockIdx.y, b = blockIdx.z, h = hq / a.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const lowram_pages& pg = a.pg;
  const int P = pg.page_tokens;
  const int seen = max(0, paged_len(pg, b, a.status) - a.n_q + j + 1);
  const size_t row = ((size_t)b * a.n_q + j) * a.Hq + hq;
  float q[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = ldf((const T*)a.q, row * D + lane * E + e) * rsqrtf((float)D);
    acc[e] = 0.f;
  }
  for (int t = warp; t < seen; t += kWarps) {
    const int page = paged_page(pg, b, t / P, a.status);
    if (page < 0) continue;
    const size_t ph = (size_t)page * a.H + h, at = (ph * P + t % P) * D + lane * E;
    float k[4], v[4];
    if (E == 4) {
      e4m3x4_to_float(*(const uint32_t*)((const uint8_t*)pg.k_code + at), k);
      e4m3x4_to_float(*(const uint32_t*)((const uint8_t*)pg.v_code + at), v);
    } else {
      e4m3x4_to_float(*(const uint16_t*)((const uint8_t*)pg.k_code + at), k);
      e4m3x4_to_float(*(const uint16_t*)((const uint8_t*)pg.v_code + at), v);
    }
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) z = fmaf(q[e], k[e], z);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    z *= pg.k_scale[ph];
    const float mn = fmaxf(m, z);
    const float c = m == -INFINITY ? 0.f : expf(m - mn);
    const float p = expf(z - mn), pv = p * pg.v_scale[ph];
    m = mn;
    l = fmaf(l, c, p);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(pv, v[e], acc[e] * c);
  }
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
  for (int w = 0; w < kWarps; ++w) L += s_m[w] == -INFINITY ? 0.f : s_l[w] * expf(s_m[w] - M);
  for (int e = threadIdx.x; e < D; e += kWarps * 32) {
    float o = 0.f;
    for (int w = 0; w < kWarps; ++w) o += s_m[w] == -INFINITY ? 0.f : s_o[w][e] * expf(s_m[w] - M);
    ((T*)a.out)[row * D + e] = from_f<T>(L > 0.f ? o / L : (L == 0.f ? 0.f : o));
  }
  if (a.lse && threadIdx.x == 0) a.lse[row] = L == 0.f ? -INFINITY : M + logf(L);
}

}  // namespace

size_t paged_attend_workspace_bytes(int, int, int, int, int, int) { return 256; }

cudaError_t launch_paged_attend(const PagedArgs& a, int, cudaStream_t s) {
  const dim3 grid(a.n_q, a.Hq, a.pg.n_seqs);
  if (a.dtype == LOWRAM_DTYPE_BF16) {
    if (a.d == 128) paged_attend_kernel<__nv_bfloat16, 128><<<grid, kWarps * 32, 0, s>>>(a);
    else paged_attend_kernel<__nv_bfloat16, 64><<<grid, kWarps * 32, 0, s>>>(a);
  } else {
    if (a.d == 128) paged_attend_kernel<float, 128><<<grid, kWarps * 32, 0, s>>>(a);
    else paged_attend_kernel<float, 64><<<grid, kWarps * 32, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace lowram
