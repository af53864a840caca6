// Paged 8-bit cache: append (rotation, scales, rounding to e4m3) and gather.
//
// Append. For the new tokens of a page and one KV head, keys and values apart:
//   x = R(pos) k (rotate-half) or v;  amax = max |x| over finite x;
//   s = smallest 2^e >= 2^-64 with amax <= 448 * 2^e;  code = e4m3_rn(x / s),
// and if the page already holds tokens of the sequence, s is at least the page's scale and the
// earlier codes are rounded again to s. With powers of two that second rounding is exact unless
// the code becomes subnormal, so it does not matter (to 2^-10 s) in how many calls a page was
// filled; a scale amax / 448 would gain nothing, since e4m3's steps are relative.
//
// Bound by bytes: 2 N H d (es + 1). One CTA takes one (page, keys or values) of a sequence and
// all heads or a share of them: a warp holds 16 rows of one head in registers, so the input is
// read once, and the (cos, sin) of the page's positions are formed once in fp64 (three table
// levels, two angle additions) into shared memory for all heads. Angles and products are fp64
// (four operations a pair) because e4m3's rounding and the scale's power of two are decisions:
// an fp32 rotation would flip one in about 2^20 of them against the formula.
#include "paged_common.cuh"

namespace lowram {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerWarp = 16;

// (cos, sin)(pos * theta_i), pos < 2^24
__device__ __forceinline__ double2 rope_any64(const RopeTables& rt, int i, int pos) {
  const double2 lo = rt.lo64[(pos & (kRopeLo - 1)) * rt.half + i];
  const double2 mi = rt.mid64[((pos >> kRopeLoBits) & ((1 << kRopeMidBits) - 1)) * rt.half + i];
  const double2 to = rt.top64[(pos >> (kRopeLoBits + kRopeMidBits)) * rt.half + i];
  const double2 hi = make_double2(to.x * mi.x - to.y * mi.y, to.y * mi.x + to.x * mi.y);
  return make_double2(hi.x * lo.x - hi.y * lo.y, hi.y * lo.x + hi.x * lo.y);
}

// exponent e of the smallest 2^e, e >= -64, with amax <= 448 * 2^e (448 = 1.75 * 2^8)
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -64 ? -64 : e;
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

template <typename T, int E> struct RowLoad;   // E consecutive elements as floats
template <> struct RowLoad<__nv_bfloat16, 4> {
  __device__ static void load(const __nv_bfloat16* p, float* o) { VecLoad<__nv_bfloat16, 4>::load(p, o); }
};
template <> struct RowLoad<__nv_bfloat16, 2> {
  __device__ static void load(const __nv_bfloat16* p, float* o) { VecLoad<__nv_bfloat16, 2>::load(p, o); }
};
template <> struct RowLoad<float, 4> {
  __device__ static void load(const float* p, float* o) { VecLoad<float, 4>::load(p, o); }
};
template <> struct RowLoad<float, 2> {
  __device__ static void load(const float* p, float* o) { VecLoad<float, 2>::load(p, o); }
};

template <int E> __device__ __forceinline__ void store_codes(uint8_t* p, const float* x);
template <> __device__ __forceinline__ void store_codes<4>(uint8_t* p, const float* x) {
  *reinterpret_cast<uint32_t*>(p) = float4_to_e4m3x4(x);
}
template <> __device__ __forceinline__ void store_codes<2>(uint8_t* p, const float* x) {
  *reinterpret_cast<uint16_t*>(p) = (uint16_t)float2_to_e4m3x2(x[0], x[1]);
}

// grid (pages of a sequence, n_seqs, 2 * head groups); dynamic shared memory: page_tokens * d/2
// double2 (rotation). Lane l of a warp: rows 2 k + (l >> 4), elements E (l & 15) .. of the row's
// first and second half.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const PagedArgs a) {
  constexpr int kHalf = D / 2, E = kHalf / 16, kRows = kRowsPerWarp / 2;
  extern __shared__ double2 s_trig[];
  __shared__ float s_amax[kThreads / 32];
  const lowram_pages& pg = a.pg;
  const int P = pg.page_tokens, b = blockIdx.y;
  const bool keys = (blockIdx.z & 1) == 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  int r0, n;
  if (a.cu_new) {
    r0 = a.cu_new[b];
    n = a.cu_new[b + 1] - r0;
    if (r0 < 0 || n < 0 || n > a.max_new || r0 > a.n_new - n) {
      if (blockIdx.x == 0 && tid == 0) raise_status(a.status, kStatusDeviceCheck);
      return;
    }
  } else {
    n = a.max_new;
    r0 = b * n;
  }
  if (n == 0) return;
  const int len = pg.lens[b], first = len - n;
  const int base = a.pos_base ? a.pos_base[b] : 0;
  if (first < 0 || len > pg.max_pages * P ||
      (a.rotate && (base < -first || base > kMaxPosition - len))) {
    if (blockIdx.x == 0 && tid == 0) raise_status(a.status, kStatusDeviceCheck);
    return;
  }
  const int pi = first / P + blockIdx.x, p0 = pi * P;   // the page's first token
  if (p0 >= len) return;
  const int page = paged_page(pg, b, pi, a.status);
  if (page < 0) return;
  const int lo = max(first, p0) - p0, hi = min(len, p0 + P) - p0;   // new rows lo .. hi-1
  const bool rotate = keys && a.rotate;
  if (rotate) {
    // a thread takes one pair and consecutive rows: the first from the tables, the others by
    // turning on by theta_i (at most 16 turns: 2^-49)
    constexpr int kPer = kThreads / kHalf;                 // threads of a pair
    const int i = tid % kHalf, rows = (hi - lo + kPer - 1) / kPer;
    const int ra = lo + (tid / kHalf) * rows, rb = min(hi, ra + rows);
    if (ra < rb) {
      const double2 d = a.rope.lo64[a.rope.half + i];      // (cos, sin)(theta_i)
      double2 c = rope_any64(a.rope, i, base + p0 + ra);
      s_trig[ra * kHalf + i] = c;
      for (int r = ra + 1; r < rb; ++r) {
        c = make_double2(c.x * d.x - c.y * d.y, c.y * d.x + c.x * d.y);
        s_trig[r * kHalf + i] = c;
      }
    }
    __syncthreads();
  }
  const T* src = (const T*)(keys ? a.k_new : a.v_new) ;
  const int64_t stride = keys ? a.k_stride : a.v_stride;
  uint8_t* codes = (uint8_t*)(keys ? pg.k_code : pg.v_code);
  float* scales = keys ? pg.k_scale : pg.v_scale;
  const int wt = P / kRowsPerWarp;                     // warps of a head's team
  const int teams = (kThreads / 32) / wt, team = warp / wt;
  const int row0 = (warp % wt) * kRowsPerWarp + (lane >> 4);
  const int el = E * (lane & 15);
  const int groups = gridDim.z >> 1, hpg = (a.H + groups - 1) / groups;
  const int h_begin = (blockIdx.z >> 1) * hpg, h_end = min(a.H, h_begin + hpg);
  for (int h0 = h_begin; h0 < h_end; h0 += teams) {
    const int h = h0 + team;
    const bool mine = h < h_end;
    float x[kRows][2 * E];
    float amax = 0.f;
    if (mine) {
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int r = row0 + 2 * k;
        if (r >= lo && r < hi) {
          const T* p = src + (int64_t)(r0 + p0 + r - first) * stride + (int64_t)h * D + el;
          RowLoad<T, E>::load(p, x[k]);
          RowLoad<T, E>::load(p + kHalf, x[k] + E);
        }
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int r = row0 + 2 * k;
        if (r >= lo && r < hi) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (rotate) {
              const double2 cs = s_trig[r * kHalf + el + e];
              const double u = x[k][e], v = x[k][E + e];
              x[k][e] = (float)(u * cs.x - v * cs.y);
              x[k][E + e] = (float)(u * cs.y + v * cs.x);
            }
          }
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) {
            const float m = fabsf(x[k][e]);
            if (m <= 3.402823466e38f) amax = fmaxf(amax, m);
            else x[k][e] = __int_as_float(0x7fffffff);   // infinities become NaN codes
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const size_t ph = (size_t)page * a.H + (mine ? h : 0);
    const float old = mine && lo > 0 ? scales[ph] : 0.f;
    if (wt > 1) {   // the team's maximum; everyone has read the old scale before it is replaced
      if (lane == 0) s_amax[warp] = amax;
      __syncthreads();
      amax = s_amax[team * wt];
      for (int w = 1; w < wt; ++w) amax = fmaxf(amax, s_amax[team * wt + w]);
      __syncthreads();
    } else {
      __syncwarp();
    }
    if (!mine) continue;
    const float fresh = pow2f(scale_exponent(amax));
    const float s = fmaxf(fresh, old);
    if (warp % wt == 0 && lane == 0) scales[ph] = s;
    uint8_t* dst = codes + ph * (size_t)P * D;
    const float inv = 1.0f / s;   // exact: a power of two between 2^-120 and 2^64
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = row0 + 2 * k;
      if (r >= lo && r < hi) {
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) x[k][e] *= inv;
        store_codes<E>(dst + r * D + el, x[k]);
        store_codes<E>(dst + r * D + kHalf + el, x[k] + E);
      }
    }
    if (lo > 0 && s > old) {   // earlier tokens of the page, at the larger scale
      const float ratio = old * inv;
      const int rw = (warp % wt) * kRowsPerWarp;
      for (int o = lane; o < kRowsPerWarp * (D / 4); o += 32) {
        const int r = rw + o / (D / 4);
        if (r >= lo) break;
        uint32_t* w = reinterpret_cast<uint32_t*>(dst + r * D) + o % (D / 4);
        float f[4];
        e4m3x4_to_float(*w, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] *= ratio;
        *w = float4_to_e4m3x4(f);
      }
    }
  }
}

// Gather. Bound by bytes: 2 B n H d (1 + es). A warp takes the rows of one page and head, keys or
// values: one look-up of page and scale, then 16-byte stores, a row's 128 or 256 bytes at a time,
// with the codes of eight stores in flight.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) paged_gather_kernel(const PagedArgs a) {
  constexpr int E = 16 / sizeof(T), kLanes = D / E;   // codes of a store, lanes of a row
  constexpr int kRows = 32 / kLanes > 0 ? 32 / kLanes : 1, kParts = kLanes > 32 ? kLanes / 32 : 1;
  const lowram_pages& pg = a.pg;
  const int P = pg.page_tokens, b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  const uint8_t* codes = (const uint8_t*)(blockIdx.z ? pg.v_code : pg.k_code);
  const float* scales = blockIdx.z ? pg.v_scale : pg.k_scale;
  T* out = (T*)(blockIdx.z ? a.v_out : a.k_out) + (size_t)b * a.n * a.H * D;
  const int len = paged_len(pg, b, a.status);
  const int64_t start = a.start ? a.start[b] : 0;
  const int64_t p0 = start >= 0 ? start / P : -((P - 1 - start) / P);   // floor
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + warp;
  const int64_t pi = p0 + unit / a.H;
  const int h = (int)(unit % a.H);
  // rows of the page inside the run
  const int64_t t0 = pi * P;
  const int lo = (int)max((int64_t)0, start - t0), hi = (int)min((int64_t)P, start + a.n - t0);
  if (lo >= hi) return;
  int page = -1;
  if (t0 + hi > 0 && t0 + lo < len && t0 >= 0) page = paged_page(pg, b, (int)pi, a.status);
  const int held = page < 0 ? 0 : (int)min((int64_t)hi, len - t0);   // rows lo .. held-1 are tokens
  const size_t ph = (size_t)(page < 0 ? 0 : page) * a.H + h;
  const float s = page < 0 ? 0.f : scales[ph];
  const uint8_t* src = codes + ph * (size_t)P * D;
  const int r0 = lane / kLanes, el = (lane % kLanes) * E;
  constexpr int kU = 8;
  for (int r = lo; r < hi; r += kU * kRows / kParts) {
    uint32_t w[kU][E / 4];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int row = r + (k / kParts) * kRows + r0, e0 = el + (k % kParts) * 32 * E;
#pragma unroll
      for (int e = 0; e < E / 4; ++e) w[k][e] = 0;
      if (row < held) {
        if constexpr (E == 8) {
          const uint2 y = *reinterpret_cast<const uint2*>(src + row * D + e0);
          w[k][0] = y.x;
          w[k][1] = y.y;
        } else {
          w[k][0] = *reinterpret_cast<const uint32_t*>(src + row * D + e0);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int row = r + (k / kParts) * kRows + r0, e0 = el + (k % kParts) * 32 * E;
      if (row >= hi) continue;
      float x[E];
      alignas(16) T y[E];
#pragma unroll
      for (int e = 0; e < E / 4; ++e) e4m3x4_to_float(w[k][e], x + 4 * e);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = from_f<T>(x[e] * s);
      *reinterpret_cast<uint4*>(out + ((size_t)(t0 + row - start) * a.H + h) * D + e0) =
          *reinterpret_cast<const uint4*>(y);
    }
  }
}

template <typename T, int D>
cudaError_t append_t(const PagedArgs& a, int num_sms, cudaStream_t s) {
  const int P = a.pg.page_tokens;
  const int64_t n_slots = ((int64_t)a.max_new + 2 * P - 2) / P;   // pages n tokens can touch
  const int teams = (kThreads / 32) / (P / kRowsPerWarp);
  const int passes = (a.H + teams - 1) / teams;
  // few CTAs: a share of the heads each; many: all heads, so that a page's angles are formed once
  const int groups = n_slots * a.pg.n_seqs * 2 * passes <= 4 * num_sms ? passes : 1;
  const size_t smem = a.rotate ? (size_t)P * (D / 2) * sizeof(double2) : 0;
  cudaError_t e = cudaFuncSetAttribute(paged_append_kernel<T, D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_append_kernel<T, D>,
                          dim3((unsigned)n_slots, a.pg.n_seqs, 2 * groups), kThreads, smem, s, a);
}

template <typename T, int D>
cudaError_t gather_t(const PagedArgs& a, cudaStream_t s) {
  const int P = a.pg.page_tokens;
  const int64_t units = ((int64_t)(a.n - 1) / P + 2) * a.H;   // pages a run can touch
  return launch_dependent(paged_gather_kernel<T, D>,
                          dim3((unsigned)((units + kThreads / 32 - 1) / (kThreads / 32)),
                               a.pg.n_seqs, 2),
                          kThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_paged_append(const PagedArgs& a, int num_sms, cudaStream_t s) {
  if (a.dtype == LOWRAM_DTYPE_BF16)
    return a.d == 128 ? append_t<__nv_bfloat16, 128>(a, num_sms, s)
                      : append_t<__nv_bfloat16, 64>(a, num_sms, s);
  return a.d == 128 ? append_t<float, 128>(a, num_sms, s) : append_t<float, 64>(a, num_sms, s);
}

cudaError_t launch_paged_gather(const PagedArgs& a, cudaStream_t s) {
  if (a.dtype == LOWRAM_DTYPE_BF16)
    return a.d == 128 ? gather_t<__nv_bfloat16, 128>(a, s)
                      : gather_t<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? gather_t<float, 128>(a, s) : gather_t<float, 64>(a, s);
}

}  // namespace lowram
