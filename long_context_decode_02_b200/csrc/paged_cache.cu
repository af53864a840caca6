// Paged 8-bit cache: append (rotation, scales, rounding to e4m3) and gather.
//
// Append. For the new tokens of a page and one KV head, keys and values apart:
//   x = R(pos) k (rotate-half) or v;  amax = max |x| over finite x;
//   s = smallest 2^e >= 2^-64 with amax <= 448 * 2^e;  code = e4m3_rn(x / s),
// and if the page already holds tokens of the sequence, s is at least the page's scale and the
// earlier codes are rounded again to s. With powers of two that second rounding is exact unless
// the code becomes subnormal, so it does not matter (to one subnormal step, 2^-9 s) in how many
// calls a page was filled; a scale amax / 448 would gain nothing, since e4m3's steps are relative.
//
// Bound by bytes: 2 N H d (es + 1). A warp takes 16 rows of one page and head, keys or values; the
// 1, 2 or 4 warps of a (page, head) agree on its maximum. A lane holds the same two pairs (four
// elements) of each of its rows in registers, so the input is read once, and turns its (cos, sin)
// on from row to row by theta_i: one look-up (four table levels) a warp, four fp64 operations a
// row and pair. Angles and products are fp64 because e4m3's rounding and the
// scale's power of two are decisions: an fp32 rotation would flip one in about 2^20 of them
// against the formula. Short-lived CTAs, five an SM, keep the loads in flight; a CTA that went
// over several (page, head)s and requested the next rows early took twice as long (112 us against
// 50 for 23.3K tokens of 8 heads, pages of 64, then; 43 now): 128 registers a thread were not
// enough for both. The number of CTAs an SM costs registers too: at d = 128 the kernels of five
// (bf16, 96 registers) and four (fp32, 128) spill 268 and 160 bytes, with four and three 36 and
// none, and were slower for it: 44.2 us against 43.4 in bf16, 55.4 against 51.1 in fp32 (d = 64,
// where neither spills: 27.0 against 24.6, 37.0 against 31.1).
#include <type_traits>

#include "paged_common.cuh"

namespace lowram {
namespace {

constexpr int kThreads = 256;        // gather
constexpr int kAppendThreads = 128;
constexpr int kRowsPerWarp = 16;

__device__ __forceinline__ double2 turn(double2 c, double2 d) {   // angles added
  return make_double2(c.x * d.x - c.y * d.y, c.y * d.x + c.x * d.y);
}
// (cos, sin)(pos * theta_i), pos < 2^24
__device__ __forceinline__ double2 rope_any64(const RopeTables& rt, int i, int pos) {
  constexpr int kFar = 1 << kRopeFarBits;
  double2 c = rt.lo64[(pos & (kRopeLo - 1)) * rt.half + i], f[kRopeFarLevels];
#pragma unroll
  for (int l = 0; l < kRopeFarLevels; ++l)
    f[l] = rt.far64[(kFar * l + ((pos >> (kRopeLoBits + kRopeFarBits * l)) & (kFar - 1))) * rt.half + i];
#pragma unroll
  for (int l = 0; l < kRopeFarLevels; ++l) c = turn(c, f[l]);
  return c;
}

// exponent e of the smallest 2^e, e >= -64, with amax <= 448 * 2^e (448 = 1.75 * 2^8)
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -64 ? -64 : e;
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// Two consecutive elements as loaded, and as floats.
template <typename T> struct Two;
template <> struct Two<__nv_bfloat16> {
  using Raw = uint32_t;
  static __device__ __forceinline__ float2 get(Raw r) { return bf2_to_f2(r); }
};
template <> struct Two<float> {
  using Raw = float2;
  static __device__ __forceinline__ float2 get(Raw r) { return r; }
};

// grid (units of a sequence / teams, n_seqs, 2): a unit is a (page, head), a team the warps of one.
// Lane l: pairs 2 (l % LR), + 1 of rows l / LR + RS k.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 2 ? 5 : 4)
paged_append_kernel(const PagedArgs a) {
  using Raw = typename Two<T>::Raw;
  constexpr int kHalf = D / 2, LR = kHalf / 2, RS = 32 / LR, NR = kRowsPerWarp / RS;
  __shared__ float s_amax[kAppendThreads / 32];
  const lowram_pages& pg = a.pg;
  const int P = pg.page_tokens, b = blockIdx.y;
  const bool keys = blockIdx.z == 0, rotate = keys && a.rotate;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  int r0, n;
  const int len = pg.lens[b], base = a.pos_base ? a.pos_base[b] : 0;
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
  const int first = len - n;
  if (first < 0 || len > pg.max_pages * P ||
      (a.rotate && (base < -first || base > kMaxPosition - len))) {
    if (blockIdx.x == 0 && tid == 0) raise_status(a.status, kStatusDeviceCheck);
    return;
  }
  const T* src = (const T*)(keys ? a.k_new : a.v_new);
  const int64_t stride = keys ? a.k_stride : a.v_stride;
  uint8_t* codes = (uint8_t*)(keys ? pg.k_code : pg.v_code);
  float* scales = keys ? pg.k_scale : pg.v_scale;
  const int wt = P / kRowsPerWarp, teams = (kAppendThreads / 32) / wt, team = warp / wt;
  const int page0 = first / P;
  const int units = ((len - 1) / P - page0 + 1) * a.H;
  if ((int)blockIdx.x * teams >= units) return;   // the whole CTA
  const int unit = blockIdx.x * teams + team;
  const bool mine = unit < units;
  const int row0 = (warp % wt) * kRowsPerWarp + lane / LR;   // this lane's first row
  const int i0 = 2 * (lane % LR);                             // its pairs i0, i0 + 1
  const int pi = page0 + unit / a.H, h = unit % a.H, p0 = pi * P;
  const int lo = max(first, p0) - p0, hi = min(len, p0 + P) - p0;   // new rows lo .. hi-1
  const int wrow = (warp % wt) * kRowsPerWarp;   // the warp's rows wrow .. wrow + 15
  const bool any = mine && wrow < hi && wrow + kRowsPerWarp > lo;
  const bool all = any && wrow >= lo && wrow + kRowsPerWarp <= hi;
  int page = mine ? pg.table[(size_t)b * pg.max_pages + pi] : -1;   // looked at further below
  float x[NR][4];   // pair i0's first and second element, pair i0 + 1's
  float amax = 0.f;
  // ROT: rotated keys. ALL: every row of the warp is new, as in all pages of a long prompt but
  // its ends (a third of the instructions are the others' comparisons).
  auto take = [&](auto rot, auto all_rows) {
    constexpr bool ROT = decltype(rot)::value, ALL = decltype(all_rows)::value;
    Raw raw[NR][2];
    const T* p = src + (int64_t)(r0 + p0 + row0 - first) * stride + (int64_t)h * D + i0;
    const int64_t step = RS * stride;
#pragma unroll
    for (int k = 0; k < NR; ++k, p += step) {
      const int r = row0 + RS * k;
      if (ALL || (r >= lo && r < hi)) {
        raw[k][0] = *reinterpret_cast<const Raw*>(p);
        raw[k][1] = *reinterpret_cast<const Raw*>(p + kHalf);
      }
    }
    double2 c[2], d[2];
    if (ROT) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // rows before the sequence's first may lie below position 0, rows behind its last above
        // the tables
        const int pos = min(base + p0 + row0, kMaxPosition - 1);
        c[e] = rope_any64(a.rope, i0 + e, pos < 0 ? -pos : pos);
        if (pos < 0) c[e].y = -c[e].y;
        d[e] = a.rope.lo64[RS * a.rope.half + i0 + e];
      }
    }
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      const int r = row0 + RS * k;
      if (ALL || (r >= lo && r < hi)) {
        const float2 u = Two<T>::get(raw[k][0]), v = Two<T>::get(raw[k][1]);
        x[k][0] = u.x;
        x[k][1] = v.x;
        x[k][2] = u.y;
        x[k][3] = v.y;
        if (ROT) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const double y = x[k][2 * e], z = x[k][2 * e + 1];
            x[k][2 * e] = (float)(y * c[e].x - z * c[e].y);
            x[k][2 * e + 1] = (float)(y * c[e].y + z * c[e].x);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(x[k][e]));   // skips NaN
      }
      if (ROT && k + 1 < NR) {
        c[0] = turn(c[0], d[0]);
        c[1] = turn(c[1], d[1]);
      }
    }
  };
  if (all) {
    if (rotate) take(std::true_type(), std::true_type());
    else take(std::false_type(), std::true_type());
  } else if (any) {
    if (rotate) take(std::true_type(), std::false_type());
    else take(std::false_type(), std::false_type());
  }
  if (!(amax <= 3.402823466e38f)) {   // infinities become NaN codes and do not count
    amax = 0.f;
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      const int r = row0 + RS * k;
      if (r >= lo && r < hi) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (fabsf(x[k][e]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(x[k][e]));
          else x[k][e] = __int_as_float(0x7fffffff);
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (mine && (page < 0 || page >= pg.n_pages)) {
    raise_status(a.status, kStatusDeviceCheck);
    page = -1;
  }
  const size_t ph = (size_t)(page < 0 ? 0 : page) * a.H + h;
  const float old = page >= 0 && lo > 0 ? scales[ph] : 0.f;
  if (wt > 1) {   // the team's maximum; everyone has read the old scale before it is replaced
    if (lane == 0) s_amax[warp] = amax;
    __syncthreads();
    amax = s_amax[team * wt];
    for (int w = 1; w < wt; ++w) amax = fmaxf(amax, s_amax[team * wt + w]);
  } else {
    __syncwarp();
  }
  if (page < 0) return;
  const float s = fmaxf(pow2f(scale_exponent(amax)), old);
  if (warp % wt == 0 && lane == 0) scales[ph] = s;
  uint8_t* dst = codes + ph * (size_t)P * D;
  const float inv = 1.0f / s;   // exact: a power of two between 2^-120 and 2^64
  uint8_t* q = dst + row0 * D + i0;
#pragma unroll
  for (int k = 0; k < NR; ++k) {
    const int r = row0 + RS * k;
    if (all || (r >= lo && r < hi)) {
      *reinterpret_cast<uint16_t*>(q + RS * k * D) =
          (uint16_t)float2_to_e4m3x2(x[k][0] * inv, x[k][2] * inv);
      *reinterpret_cast<uint16_t*>(q + RS * k * D + kHalf) =
          (uint16_t)float2_to_e4m3x2(x[k][1] * inv, x[k][3] * inv);
    }
  }
  if (lo > 0 && s > old) {   // earlier tokens of the page, at the larger scale
    const float ratio = old * inv;
    for (int o = lane; o < kRowsPerWarp * (D / 4); o += 32) {
      const int r = wrow + o / (D / 4);
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

// Gather. Bound by bytes: 2 B n H d (1 + es). A warp takes the rows of one page and head, keys or
// values: one look-up of page and scale, then 16-byte stores, a row's 128 or 256 bytes at a time,
// with the codes of eight stores in flight: 4K tokens of 8 sequences in 32 us, 0.88 of the copy
// rate (45 with 16 codes and a look-up a thread).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) paged_gather_kernel(const PagedArgs a) {
  constexpr int E = 16 / sizeof(T), kLanes = D / E;   // codes of a store, lanes of a row
  constexpr int kRows = 32 / kLanes;                  // rows of a warp's store
  const lowram_pages& pg = a.pg;
  const int P = pg.page_tokens, b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
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
  for (int r = lo; r < hi; r += kU * kRows) {
    uint32_t w[kU][E / 4];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int row = r + k * kRows + r0;
#pragma unroll
      for (int e = 0; e < E / 4; ++e) w[k][e] = 0;
      if (row < held) {
        if constexpr (E == 8) {
          const uint2 y = *reinterpret_cast<const uint2*>(src + row * D + el);
          w[k][0] = y.x;
          w[k][1] = y.y;
        } else {
          w[k][0] = *reinterpret_cast<const uint32_t*>(src + row * D + el);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int row = r + k * kRows + r0;
      if (row >= hi) continue;
      float x[E];
      alignas(16) T y[E];
#pragma unroll
      for (int e = 0; e < E / 4; ++e) e4m3x4_to_float(w[k][e], x + 4 * e);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = from_f<T>(x[e] * s);
      *reinterpret_cast<uint4*>(out + ((size_t)(t0 + row - start) * a.H + h) * D + el) =
          *reinterpret_cast<const uint4*>(y);
    }
  }
}

template <typename T, int D>
cudaError_t append_t(const PagedArgs& a, cudaStream_t s) {
  const int P = a.pg.page_tokens;
  const int64_t units = ((int64_t)a.max_new + 2 * P - 2) / P * a.H;   // (page, head)s of n tokens
  const int teams = (kAppendThreads / 32) / (P / kRowsPerWarp);
  return launch_dependent(paged_append_kernel<T, D>,
                          dim3((unsigned)((units + teams - 1) / teams), a.pg.n_seqs, 2), kAppendThreads,
                          0, s, a);
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

cudaError_t launch_paged_append(const PagedArgs& a, cudaStream_t s) {
  if (a.dtype == LOWRAM_DTYPE_BF16)
    return a.d == 128 ? append_t<__nv_bfloat16, 128>(a, s)
                      : append_t<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? append_t<float, 128>(a, s) : append_t<float, 64>(a, s);
}

cudaError_t launch_paged_gather(const PagedArgs& a, cudaStream_t s) {
  if (a.dtype == LOWRAM_DTYPE_BF16)
    return a.d == 128 ? gather_t<__nv_bfloat16, 128>(a, s)
                      : gather_t<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? gather_t<float, 128>(a, s) : gather_t<float, 64>(a, s);
}

}  // namespace lowram
