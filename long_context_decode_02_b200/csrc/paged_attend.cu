// Attention over the paged 8-bit cache for the last n_q tokens of every sequence:
//   z_t = (q . k_code_t) k_scale / sqrt(d),  out = sum_t softmax(z)_t v_code_t v_scale.
//
// Bound by bytes: each code is read once (2 sum(len) H d bytes), for 4 G n_q operations a pair
// of codes. The work is cut into steps of 32 tokens of one (sequence, KV head, group of query
// rows); all steps in one list, an equal run of them for every warp of the GPU, so ragged
// batches and single long sequences fill it alike. A warp streams its run alone: it issues TMA
// boxes of 16 tokens into its own ring of stages, holds the queries as matrix fragments in
// registers, and writes one partial (reference, sum, output) for every (sequence, head, group)
// that its run touches. A second kernel merges the partials of a row.
//
// Matrix form, m16n8k16 with fp16 operands and fp32 sums: S^T = K Q^T (rows: 16 tokens, columns:
// 8 query rows) and O^T += V^T P^T (rows: 16 elements of d), so the 4 or 8 query rows of a KV
// head fill the narrow side and no half of a tile is idle. e4m3 codes widen to fp16 exactly
// (cvt.e4m3x2) on their way from shared memory to the fragment; which element of d or which
// token a fragment's row or k index means is free as long as both operands agree, so K comes by
// ldmatrix (a 16-byte chunk of a row is one k16 step) and V by 16- or 8-byte loads, without bank
// conflicts in the TMA swizzle. At these shapes the warps issue a third of the instruction slots
// that the bytes leave, so the tensor rate does not bound.
//
// Numbers. A query row is scaled by a power of two to a largest magnitude in [2^12, 2^13) and
// held in fp16: exact for bf16 rows (elements 2^-27 below the row's largest lose digits); fp32
// rows take two columns, fp16(q) and fp16(q - fp16(q)), whose products add up. Scores, the
// softmax's reference and sum and the output are fp32. A weight is rounded to fp16 (2^-11, eight
// times finer than the bf16 output), for fp32 again in two columns. Values carry their page's
// scale s_v = fr 2^ev inside the weight: the reference of a row is max(z + ev) over its tokens, so
//   a = 2^(z + ev - m) <= 1,  weight = a fr 2^13,  sum += a 2^-ev,
// and pages whose scales lie far apart cost each other no digits.
#include <cuda.h>

#include "paged_common.cuh"
#include "sm100_ptx.cuh"

namespace lowram {
namespace {

using namespace sm100;

constexpr int kWarps = 8;
constexpr int kStep = 32;                 // tokens of a step: two TMA boxes of 16
constexpr int kUnit = 16;
constexpr int kMaxCtas = 160;             // bound of the workspace; the grid is one CTA an SM
constexpr uint32_t kRingBytes = 24 * 1024;   // a warp's ring
constexpr float kWeightScale = 8192.f;    // 2^13: weights in fp16 stay normal down to 2^-27
constexpr int kCombineThreads = 128;

template <int D> struct Tile {
  static constexpr uint32_t kHalf = kStep * D;          // bytes of K (or V) of a step
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr int kStages = kRingBytes / kStage;   // 3 (d = 128), 6 (d = 64)
};

struct AttendMaps {
  CUtensorMap k;   // [n_pages * H * page_tokens rows][d] bytes, box d x 16, swizzled by d bytes
  CUtensorMap v;
};

// Query rows of one (sequence, KV head): r = j G + g, in groups of `rows`.
struct RowPlan {
  int rows, groups;   // rows of a group (8 or 16; fp32: 4 or 8), groups
};
__host__ __device__ inline RowPlan row_plan(int G, int n_q, int dtype) {
  const int R = G * n_q, per = dtype == LOWRAM_DTYPE_BF16 ? 8 : 4;
  RowPlan p;
  p.rows = R <= per ? per : 2 * per;
  p.groups = (R + p.rows - 1) / p.rows;
  return p;
}

// Workspace: plan { share, prefix[n_seqs + 1] } in steps, then the partials' (m, l) and outputs.
// The partial of warp w for pair x (= (b H + h) groups + group) is number w + x: both only grow
// along the list of steps.
struct AttendWs {
  long long* plan;
  float2* ml;   // [slots][rows]
  float* o;     // [slots][rows][d]
};
__host__ __device__ inline size_t ws_align(size_t x) { return (x + 255) / 256 * 256; }
inline size_t ws_slots(int H, int groups, int n_seqs) {
  return (size_t)kMaxCtas * kWarps + (size_t)n_seqs * H * groups;
}
inline AttendWs ws_layout(void* ws, int H, const RowPlan& rp, int d, int n_seqs, size_t* total) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  const size_t slots = ws_slots(H, rp.groups, n_seqs);
  size_t o = 0;
  AttendWs w;
  w.plan = reinterpret_cast<long long*>(p + o);
  o = ws_align(o + (size_t)(n_seqs + 2) * sizeof(long long));
  w.ml = reinterpret_cast<float2*>(p + o);
  o = ws_align(o + slots * rp.rows * sizeof(float2));
  w.o = reinterpret_cast<float*>(p + o);
  o = ws_align(o + slots * rp.rows * d * sizeof(float));
  if (total) *total = o;
  return w;
}

struct AttendParams {
  PagedArgs a;
  RowPlan rp;
  AttendWs ws;
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float round_f16(float x) { return __half2float(__float2half_rn(x)); }
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr) : "memory");
  return r;
}

// Token (within 8) of fragment row x. For 64-byte rows the four lanes that read together take
// rows 0, 1, 4, 5 (then 2, 3, 6, 7), which the 64-byte swizzle puts into different banks.
template <int D> __device__ __forceinline__ constexpr int tau(int x) {
  return D == 128 ? x : ((x >> 1) & 1) | ((x & 1) << 1) | ((x >> 2) << 2);
}
template <int D> __device__ __forceinline__ uint32_t chunk_offset(int row, int c) {
  return D == 128 ? sw128_offset(row, c) : sw64_offset(row, c);
}

// bit i of the result: byte i of w is a NaN code
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= ((w >> (8 * i)) & 127u) == 127u ? 1u << i : 0u;
  return r;
}

// NT: column tiles of 8. F32: a query row is two columns (high and low fp16 parts).
template <typename T, int D, int NT, bool F32>
__global__ void __launch_bounds__(kWarps * 32, 1)
paged_attend_kernel(const AttendParams p, const __grid_constant__ AttendMaps maps) {
  using TL = Tile<D>;
  constexpr int S = TL::kStages, kChunks = D / 16, kOT = D / 16, DG = D / 8;
  constexpr int CC = F32 ? 1 : 2;           // query rows of a lane in a column tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ float4 s_meta[kWarps][S][2];   // a unit: k_scale, fr 2^13, ev, valid tokens
  __shared__ alignas(8) uint64_t s_bar[kWarps][S];
  __shared__ int s_abort;
  const PagedArgs& a = p.a;
  const lowram_pages& pg = a.pg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int P = pg.page_tokens, upp = P / kUnit;      // 16-token units of a page
  const int pairs = a.H * p.rp.groups;                // of one sequence
  const int R = a.G * a.n_q;
  const uint32_t ring = ((smem_u32(smem_raw) + 1023u) & ~1023u) + warp * kRingBytes;
  if (threadIdx.x == 0) s_abort = 0;
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(smem_u32(&s_bar[warp][i]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  volatile int* abort_flag = &s_abort;

  // ---- this warp's run of steps
  long long total = 0;
  for (int b0 = 0; b0 < pg.n_seqs; b0 += 32) {
    const int b = b0 + lane;
    int n = b < pg.n_seqs ? (paged_len(pg, b, a.status) + kStep - 1) / kStep : 0;
    n = __reduce_add_sync(0xffffffffu, n);
    total += n;
  }
  total *= pairs;
  const int n_warps = gridDim.x * kWarps;
  // consecutive runs go to different SMs, so that little work still uses many of them
  const int w = warp * gridDim.x + blockIdx.x;
  const long long share = total > 0 ? (total + n_warps - 1) / n_warps : 1;
  const long long w0 = min(total, w * share), w1 = min(total, w0 + share);
  const int n_steps = (int)(w1 - w0);
  if (w == 0) {   // the plan, for the merge
    long long at = 0;
    for (int b0 = 0; b0 < pg.n_seqs; b0 += 32) {
      const int b = b0 + lane;
      const int n = b < pg.n_seqs ? (paged_len(pg, b, nullptr) + kStep - 1) / kStep : 0;
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < pg.n_seqs) p.ws.plan[1 + b] = (at + x - n) * pairs;
      at += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      p.ws.plan[0] = share;
      p.ws.plan[1 + pg.n_seqs] = total;
    }
  }
  if (n_steps == 0) return;
  // where the run begins: sequence, pair, step
  int b = 0, len = 0, ns = 0, pair = 0, step = 0;
  {
    long long at = 0;
    for (int b0 = 0;; b0 += 32) {
      const int bb = b0 + lane;
      const int n = bb < pg.n_seqs ? paged_len(pg, bb, nullptr) : 0;
      const int s = (n + kStep - 1) / kStep;
      int x = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, (at + x) * pairs > w0);
      if (past) {
        const int src = __ffs(past) - 1;
        b = b0 + src;
        len = __shfl_sync(0xffffffffu, n, src);
        ns = (len + kStep - 1) / kStep;
        const long long off = w0 - (at + __shfl_sync(0xffffffffu, x, src) - ns) * pairs;
        pair = (int)(off / ns);
        step = (int)(off % ns);
        break;
      }
      at += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  // the loader's cursor runs ahead of the consumer's
  int lb = b, llen = len, lns = ns, lpair = pair, lstep = step;
  int ubase = -1;                    // first unit of the lanes' page entries, -1: none loaded
  int upage = -1;                    // this lane's unit: page (or -1), scales
  float usk = 0.f, usv = 0.f;
  auto next_seq = [&](int& bb, int& ll, int& nn) {
    do {
      ++bb;
      ll = bb < pg.n_seqs ? paged_len(pg, bb, nullptr) : 0;
      nn = (ll + kStep - 1) / kStep;
    } while (nn == 0 && bb < pg.n_seqs);
  };
  auto issue = [&](int i) {
    const int st = i % S, u0 = 2 * lstep, h = lpair / p.rp.groups;
    if (ubase < 0 || u0 < ubase || u0 + 2 > ubase + 32) {   // the next 32 units' pages
      ubase = u0;
      const int u = u0 + lane;
      upage = -1;
      if (u * kUnit < llen) {
        upage = paged_page(pg, lb, u / upp, a.status);
        if (upage >= 0) {
          const size_t ph = (size_t)upage * a.H + h;
          usk = pg.k_scale[ph];
          usv = pg.v_scale[ph];
        }
      }
    }
    const int mine = lane - (u0 - ubase);
    const bool owner = mine == 0 || mine == 1;
    const unsigned have = __ballot_sync(0xffffffffu, owner && upage >= 0);
    const uint32_t bar = smem_u32(&s_bar[warp][st]);
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)__popc(have) * 2 * kUnit * D);
    __syncwarp();
    if (owner) {
      const int u = u0 + mine;
      if (upage >= 0) {
        const uint32_t dst = ring + st * TL::kStage + mine * kUnit * D;
        const int y = (upage * a.H + h) * P + (u % upp) * kUnit;
        tma_load_2d(dst, &maps.k, 0, y, bar);
        tma_load_2d(dst + TL::kHalf, &maps.v, 0, y, bar);
      }
      int ev = (int)((__float_as_uint(usv) >> 23) & 255u) - 127;
      ev = min(max(ev, -64), 120);
      const int valid = upage >= 0 ? min(max(llen - u * kUnit, 0), kUnit) : 0;
      s_meta[warp][st][mine] =
          make_float4(usk, usv * __int_as_float((127 - ev) << 23) * kWeightScale,
                      __int_as_float(ev), __int_as_float(valid));
    }
    if (++lstep == lns) {
      lstep = 0;
      ubase = -1;
      if (++lpair == pairs) {
        lpair = 0;
        next_seq(lb, llen, lns);
      }
    }
  };

  // ---- state of the current (sequence, head, group)
  uint32_t qf[NT][kChunks][2];
  float cs[NT][CC];                 // logit of a column in log2 units per unit of S
  int lim[NT][CC];                  // tokens a query row sees
  float m[NT][CC], l[NT][CC], O[NT][kOT][4];
  bool fresh = true, good = true;
  int landed = 0, issued = 0;
  for (int it = 0; it < n_steps + S; ++it) {
    if (it >= S) {
      const int i = it - S, st = i % S;
      const int h = pair / p.rp.groups, row0 = (pair % p.rp.groups) * p.rp.rows;
      if (fresh) {   // the group's queries
        fresh = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = row0 + (F32 ? nt * 4 + (g >> 1) : nt * 8 + g);   // this lane's column
          float x[kChunks][4], top = 0.f;
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[c][e] = 0.f;
          if (r < R) {
            const T* q = (const T*)a.q +
                         (((size_t)b * a.n_q + r / a.G) * a.Hq + h * a.G + r % a.G) * D + 4 * t;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) VecLoad<T, 4>::load(q + 16 * c, x[c]);
          }
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(x[c][e]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          int ex = (int)(__float_as_uint(top) >> 23) - 127;
          ex = min(max(ex, -100), 127);
          const float up = __int_as_float((12 - ex + 127) << 23);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[e] = x[c][e] * up;
              if (F32 && (g & 1)) y[e] -= round_f16(y[e]);
            }
            qf[nt][c][0] = pack_f16x2(y[0], y[1]);
            qf[nt][c][1] = pack_f16x2(y[2], y[3]);
          }
          const float scale = __int_as_float((ex - 12 + 127) << 23) *
                              (1.4426950408889634f * rsqrtf((float)D));
#pragma unroll
          for (int cc = 0; cc < CC; ++cc) {
            cs[nt][cc] = __shfl_sync(0xffffffffu, scale, 4 * (2 * t + cc));
            const int rr = row0 + (F32 ? nt * 4 + t : nt * 8 + 2 * t + cc);
            lim[nt][cc] = rr < R ? len - a.n_q + rr / a.G + 1 : 0;
            m[nt][cc] = -INFINITY;
            l[nt][cc] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < kOT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[nt][j][e] = 0.f;
        }
      }
      good = good && mbar_wait_bounded(smem_u32(&s_bar[warp][st]), (uint32_t)((i / S) & 1), abort_flag);
      good = __all_sync(0xffffffffu, good);
      if (!good) break;
      landed = i + 1;
      const uint32_t kb = ring + st * TL::kStage, vb = kb + TL::kHalf;
      const float4 me0 = s_meta[warp][st][0], me1 = s_meta[warp][st][1];
      const float4 me[2] = {me0, me1};
      // every token of the step is seen by every row of the group
      const bool full = __float_as_int(me0.w) == kUnit && __float_as_int(me1.w) == kUnit &&
                        (step + 1) * kStep <= len - a.n_q + row0 / a.G + 1;
      // S^T = K Q^T
      float z[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[u][nt][e] = 0.f;
        const int krow = u * kUnit + tau<D>(lane & 7) + (lane & 8);
#pragma unroll
        for (int c = 0; c < kChunks; c += 2) {
          uint32_t r[4], f[4];
          ldmatrix_x4(kb + chunk_offset<D>(krow, c + (lane >> 4)), r);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            f[0] = e4m3x2_to_f16x2((uint16_t)(r[2 * k] & 0xffffu));
            f[1] = e4m3x2_to_f16x2((uint16_t)(r[2 * k + 1] & 0xffffu));
            f[2] = e4m3x2_to_f16x2((uint16_t)(r[2 * k] >> 16));
            f[3] = e4m3x2_to_f16x2((uint16_t)(r[2 * k + 1] >> 16));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(z[u][nt], f, qf[nt][c + k][0], qf[nt][c + k][1]);
          }
        }
      }
      // logits in log2 units; masked ones -inf
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (F32 && (e & 1)) continue;
            const int cc = F32 ? 0 : e & 1;
            float x = F32 ? z[u][nt][e] + z[u][nt][e + 1] : z[u][nt][e];
            x *= cs[nt][cc] * me[u].x;
            if (!full) {
              const int tk = tau<D>(g) + (e >= 2 ? 8 : 0);
              const bool seen = tk < __float_as_int(me[u].w) &&
                                step * kStep + u * kUnit + tk < lim[nt][cc];
              x = seen ? x : -INFINITY;
            }
            z[u][nt][e] = x;
          }
      // reference: max of z + ev
      const float ev[2] = {(float)__float_as_int(me0.z), (float)__float_as_int(me1.z)};
      float mn[NT][CC];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int cc = 0; cc < CC; ++cc) {
          float x = fmaxf(fmaxf(z[0][nt][cc], z[0][nt][cc + 2]) + ev[0],
                          fmaxf(z[1][nt][cc], z[1][nt][cc + 2]) + ev[1]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          mn[nt][cc] = fmaxf(m[nt][cc], x);
          grow = grow || mn[nt][cc] > m[nt][cc];
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float corr[2];
#pragma unroll
          for (int cc = 0; cc < CC; ++cc) {
            corr[cc] = mn[nt][cc] > m[nt][cc] ? ex2_approx(m[nt][cc] - mn[nt][cc]) : 1.f;
            m[nt][cc] = mn[nt][cc];
            l[nt][cc] *= corr[cc];
          }
          if (F32) corr[1] = corr[0];
#pragma unroll
          for (int j = 0; j < kOT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[nt][j][e] *= corr[e & 1];
        }
      }
      // weights, as the B operand of O^T += V^T P^T
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float back = __int_as_float((127 - __float_as_int(me[u].z)) << 23);   // 2^-ev
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float wgt[4];
#pragma unroll
          for (int cc = 0; cc < CC; ++cc) {
            const float off = m[nt][cc] == -INFINITY ? 0.f : ev[u] - m[nt][cc];
            const float a0 = ex2_approx(z[u][nt][cc] + off), a1 = ex2_approx(z[u][nt][cc + 2] + off);
            l[nt][cc] = fmaf(a0 + a1, back, l[nt][cc]);
            wgt[cc] = a0 * me[u].y;
            wgt[cc + 2] = a1 * me[u].y;
          }
          if (F32) {
            wgt[1] = wgt[0] - round_f16(wgt[0]);
            wgt[3] = wgt[2] - round_f16(wgt[2]);
          }
          pf[u][nt][0] = movmatrix_trans(pack_f16x2(wgt[0], wgt[1]));
          pf[u][nt][1] = movmatrix_trans(pack_f16x2(wgt[2], wgt[3]));
        }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        constexpr int kW = D / 32;          // 32-bit words of a lane's share of a row
        const int ta = tau<D>(2 * t), tb = tau<D>(2 * t + 1);
        const int tok[4] = {ta, tb, ta + 8, tb + 8};
        uint32_t v[4][kW];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = u * kUnit + tok[x];
          if (D == 128) {
            const uint4 y = lds128(vb + sw128_offset(row, g));
            v[x][0] = y.x; v[x][1] = y.y;
            if (kW == 4) { v[x][kW - 2] = y.z; v[x][kW - 1] = y.w; }
          } else {
            const uint2 y = lds64(vb + sw64_offset(row, g >> 1) + 8 * (g & 1));
            v[x][0] = y.x; v[x][1] = y.y;
          }
        }
        uint32_t bad[4] = {0, 0, 0, 0};   // NaN codes of tokens that only some rows see
        bool any_bad = false;
        if (!full) {
          const int vis = len - a.n_q + row0 / a.G + 1;   // tokens that every row sees
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int tk = step * kStep + u * kUnit + tok[x];
            if (tok[x] >= __float_as_int(me[u].w)) {      // not a token: the bytes may be anything
#pragma unroll
              for (int y = 0; y < kW; ++y) v[x][y] = 0;
            } else if (tk >= vis) {
#pragma unroll
              for (int y = 0; y < kW; ++y) {
                const uint32_t nb = nan_bytes(v[x][y]);
                bad[x] |= nb << (4 * y);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (nb >> k & 1) v[x][y] &= ~(255u << (8 * k));
              }
              any_bad = any_bad || bad[x] != 0;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kOT; ++j) {
          const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
          const uint32_t x0 = __byte_perm(v[0][j / 2], v[1][j / 2], sel);
          const uint32_t x1 = __byte_perm(v[2][j / 2], v[3][j / 2], sel);
          uint32_t f[4];
          f[0] = e4m3x2_to_f16x2((uint16_t)(x0 & 0xffffu));
          f[1] = e4m3x2_to_f16x2((uint16_t)(x0 >> 16));
          f[2] = e4m3x2_to_f16x2((uint16_t)(x1 & 0xffffu));
          f[3] = e4m3x2_to_f16x2((uint16_t)(x1 >> 16));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(O[nt][j], f, pf[u][nt][0], pf[u][nt][1]);
        }
        if (__any_sync(0xffffffffu, any_bad)) {   // a NaN value reaches the rows that see it
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int src = 0; src < 4; ++src) {
              const uint32_t bits = __shfl_sync(0xffffffffu, bad[x], 4 * g + src);
              const int tx = tau<D>(2 * src + (x & 1)) + (x >= 2 ? 8 : 0);
              const int tk = step * kStep + u * kUnit + tx;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int cc = 0; cc < CC; ++cc)
                  if (tk < lim[nt][cc]) {
#pragma unroll
                    for (int j = 0; j < kOT; ++j) {
                      if (bits >> (2 * j) & 1) O[nt][j][cc] = __int_as_float(0x7fffffff);
                      if (bits >> (2 * j + 1) & 1) O[nt][j][cc + 2] = __int_as_float(0x7fffffff);
                    }
                  }
            }
        }
      }
      // end of the pair, or of the run: its partial
      const bool last = ++step == ns;
      if (last || i == n_steps - 1) {
        const size_t slot = (size_t)w + (size_t)b * pairs + pair;
        float* po = p.ws.o + slot * p.rp.rows * D;
        float2* pml = p.ws.ml + slot * p.rp.rows;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int cc = 0; cc < CC; ++cc) {
            float x = l[nt][cc];
            x += __shfl_xor_sync(0xffffffffu, x, 4);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            const int r = F32 ? nt * 4 + t : nt * 8 + 2 * t + cc;   // row of the group
            if (row0 + r < R) {
              if (g == 0) pml[r] = make_float2(m[nt][cc], x);
#pragma unroll
              for (int j = 0; j < kOT; ++j) {
                float2 o = make_float2(O[nt][j][cc], O[nt][j][cc + 2]);
                if (F32) o = make_float2(O[nt][j][0] + O[nt][j][1], O[nt][j][2] + O[nt][j][3]);
                *reinterpret_cast<float2*>(po + (size_t)r * D + DG * g + 2 * j) = o;
              }
            }
          }
        fresh = true;
        if (last) {
          step = 0;
          if (++pair == pairs) {
            pair = 0;
            next_seq(b, len, ns);
          }
        }
      }
    }
    __syncwarp();   // every lane has read the stage (and its meta) that is filled again
    if (it < n_steps) {
      issue(it);
      issued = it + 1;
    }
  }
  if (!good) {   // a wait gave up: the copies still in flight land first
    if (lane == 0) raise_status(a.status, kStatusTimeout);
    for (int i = landed; i < issued; ++i) {
      int dummy = 0;
      mbar_wait_bounded(smem_u32(&s_bar[warp][i % S]), (uint32_t)((i / S) & 1), &dummy);
    }
  }
}

// One CTA a query row: out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s over the partials
// of its pair; the warps take every fourth partial.
template <typename T, int D>
__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const AttendParams p) {
  constexpr int E = D / 32, kW = kCombineThreads / 32;
  const PagedArgs& a = p.a;
  const int hq = blockIdx.x % a.Hq, j = blockIdx.x / a.Hq, b = blockIdx.y;
  const int h = hq / a.G, r = j * a.G + hq % a.G;
  const int grp = r / p.rp.rows, rg = r % p.rp.rows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = a.H * p.rp.groups, pair = h * p.rp.groups + grp;
  const long long share = p.ws.plan[0];
  const long long begin = p.ws.plan[1 + b], ns = (p.ws.plan[2 + b] - begin) / pairs;
  const size_t row = ((size_t)b * a.n_q + j) * a.Hq + hq;
  const long long s0 = begin + pair * ns;
  const int first = (int)(s0 / share);
  const int count = ns > 0 ? (int)((s0 + ns - 1) / share) - first + 1 : 0;
  const size_t slot0 = (size_t)first + (size_t)b * pairs + pair;
  const float2* ml = p.ws.ml + slot0 * p.rp.rows + rg;
  const float* po = p.ws.o + (slot0 * p.rp.rows + rg) * D + lane * E;
  const size_t so = (size_t)p.rp.rows * D;
  float M = -INFINITY;
  for (int s = lane; s < count; s += 32) M = fmaxf(M, ml[(size_t)s * p.rp.rows].x);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int s = warp; s < count; s += kW) {
    const float2 x = ml[(size_t)s * p.rp.rows];
    // a partial that saw nothing holds zeros; a NaN sum must stay one
    const float c = x.x == -INFINITY ? (x.y == 0.f ? 0.f : 1.f) : exp2f(x.x - M);
    L = fmaf(c, x.y, L);
    float o[E];
    if (E == 4) {
      const float4 y = *reinterpret_cast<const float4*>(po + s * so);
      o[0] = y.x; o[1] = y.y; o[E - 2] = y.z; o[E - 1] = y.w;
    } else {
      const float2 y = *reinterpret_cast<const float2*>(po + s * so);
      o[0] = y.x; o[1] = y.y;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(c, o[e], acc[e]);
  }
  __shared__ float s_l[kW], s_o[kW][D];
  if (lane == 0) s_l[warp] = L;
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int x = 0; x < kW; ++x) L += s_l[x];
  const float inv = L == 0.f ? 0.f : 1.f / (L * kWeightScale);
  for (int e = threadIdx.x; e < D; e += kCombineThreads) {
    float o = 0.f;
#pragma unroll
    for (int x = 0; x < kW; ++x) o += s_o[x][e];
    ((T*)a.out)[row * D + e] = from_f<T>(o * inv);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[row] = L == 0.f ? -INFINITY : fmaf(M, 0.69314718055994531f, logf(L));
}

template <typename T, int D, int NT, bool F32>
cudaError_t attend_t(const AttendParams& p, int num_sms, cudaStream_t s) {
  const PagedArgs& a = p.a;
  AttendMaps maps;
  const uint64_t rows = (uint64_t)a.pg.n_pages * a.H * a.pg.page_tokens;
  if (!make_tensor_map_2d(&maps.k, a.pg.k_code, kMapBytes, D, rows, D, kUnit, D, 256) ||
      !make_tensor_map_2d(&maps.v, a.pg.v_code, kMapBytes, D, rows, D, kUnit, D, 256))
    return cudaErrorInvalidValue;
  const size_t smem = (size_t)kWarps * kRingBytes + 1024;
  auto kern = paged_attend_kernel<T, D, NT, F32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<num_sms < kMaxCtas ? num_sms : kMaxCtas, kWarps * 32, smem, s>>>(p, maps);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  paged_combine_kernel<T, D><<<dim3(a.n_q * a.Hq, a.pg.n_seqs), kCombineThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int D, bool F32>
cudaError_t attend_d(const AttendParams& p, int num_sms, cudaStream_t s) {
  return p.rp.rows == (F32 ? 4 : 8) ? attend_t<T, D, 1, F32>(p, num_sms, s)
                                    : attend_t<T, D, 2, F32>(p, num_sms, s);
}

}  // namespace

size_t paged_attend_workspace_bytes(int H, int G, int d, int dtype, int n_seqs, int n_q) {
  size_t total = 0;
  ws_layout(nullptr, H, row_plan(G, n_q, dtype), d, n_seqs, &total);
  return total;
}

cudaError_t launch_paged_attend(const PagedArgs& a, int num_sms, cudaStream_t s) {
  AttendParams p{};
  p.a = a;
  p.rp = row_plan(a.G, a.n_q, a.dtype);
  p.ws = ws_layout(a.ws, a.H, p.rp, a.d, a.pg.n_seqs, nullptr);
  if (a.dtype == LOWRAM_DTYPE_BF16)
    return a.d == 128 ? attend_d<__nv_bfloat16, 128, false>(p, num_sms, s)
                      : attend_d<__nv_bfloat16, 64, false>(p, num_sms, s);
  return a.d == 128 ? attend_d<float, 128, true>(p, num_sms, s)
                    : attend_d<float, 64, true>(p, num_sms, s);
}

}  // namespace lowram
