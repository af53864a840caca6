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
// Matrix form, m16n8k16 with fp16 operands and fp32 sums: S^T = K Q^T (rows: 16 tokens) and
// O^T += V^T P^T (rows: 16 elements of d), so the few query rows of a KV head fill the narrow side
// of 8 columns. e4m3 codes widen to fp16 exactly on their way from shared memory to the
// fragment: K comes by ldmatrix (a 16-byte chunk of a row is one k16 step; which element of d a k
// index means is free as long as the queries agree), V by ldmatrix's transposing 8-bit form, both
// without bank conflicts in the TMA swizzle. (e4m3 operands in mma.sync take no conversion in the
// source but cost three times the instructions here: 706 a step of 32 tokens.)
//
// Numbers. A query row is scaled by a power of two to a largest magnitude in [2^12, 2^13) and
// held in fp16: exact for bf16 rows (elements 2^-27 below the row's largest lose digits); fp32
// rows take two columns, fp16(q) and fp16(q - fp16(q)), whose products add up to 2^-22. Scores,
// the softmax's reference and sum and the output are fp32. A weight is rounded to fp16 (2^-11,
// eight times finer than the bf16 output), for fp32 again in two columns (2^-22). The matrix
// unit cuts its sums toward zero, so fp32 contexts start each step's product from zero and add it
// to the output in fp32: a cut of 2^-24 for each of a run's thousands of tokens is a bias of 1e-6.
// Values carry their page's scale s_v = fr 2^ev inside the weight: the reference of a row is
// max(z + ev) over its tokens, so
//   a = 2^(z + ev - m) <= 1,  weight = a fr 2^13,  sum += a 2^-ev,
// and pages whose scales lie far apart cost each other no digits.
#include <cuda.h>

#include "paged_common.cuh"
#include "sm100_ptx.cuh"

namespace lowram {
namespace {

using namespace sm100;

constexpr int kWarps = 8;
constexpr int kStep = 32;                 // tokens of a step: two units
constexpr int kUnit = 16;
constexpr int kMetaUnits = 64;            // a warp's ring of units' scales
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
  CUtensorMap k;   // [n_pages * H * page_tokens rows][d] bytes, box d x min(page_tokens, 32),
                   // swizzled by d bytes
  CUtensorMap v;
};

// Query rows of one (sequence, KV head): r = j G + g, in groups of `rows`.
struct RowPlan {
  int rows, groups;   // rows of a group (4 or 8), groups
};
inline RowPlan row_plan(int G, int n_q) {
  const int R = G * n_q;
  RowPlan p;
  p.rows = R <= 4 ? 4 : 8;
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
inline size_t ws_align(size_t x) { return (x + 255) / 256 * 256; }
inline AttendWs ws_layout(void* ws, int H, const RowPlan& rp, int d, int n_seqs, size_t* total) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  const size_t slots = (size_t)kMaxCtas * kWarps + (size_t)n_seqs * H * rp.groups;
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
// Two 16 x 16 byte matrices, rows named by lanes 0-15 and 16-31: lane (g, t) gets column g of
// rows 4 t .. 4 t + 3 of the first (r[0]), column g + 8 (r[1]), and the second's (r[2], r[3]).
__device__ __forceinline__ void ldmatrix_b8_trans(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
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
__device__ __forceinline__ void mma_f16_first(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Fragment of codes: bytes 0, 1 of w0 and w1, then bytes 2, 3.
__device__ __forceinline__ void widen(uint32_t w0, uint32_t w1, uint32_t* f) {
  f[0] = e4m3x2_to_f16x2((uint16_t)(w0 & 0xffffu));
  f[1] = e4m3x2_to_f16x2((uint16_t)(w1 & 0xffffu));
  f[2] = e4m3x2_to_f16x2((uint16_t)(w0 >> 16));
  f[3] = e4m3x2_to_f16x2((uint16_t)(w1 >> 16));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float round_f16(float x) { return __half2float(__float2half_rn(x)); }

// Token (of 16) of fragment row x of S^T, and of row r that ldmatrix transposes for V. The two
// agree: a fragment of P^T has rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of S^T in lane t, and the V
// fragment takes them from rows 4 t .. 4 t + 3. Any eight rows that ldmatrix reads together lie in
// different residues of 8: no bank conflict.
__device__ __forceinline__ int s_token(int x) { return x < 8 ? x : 8 + ((x + 4) & 7); }
__device__ __forceinline__ int v_token(int r) {
  return s_token(2 * (r >> 2) + (r & 1) + ((r & 2) << 2));
}
template <int D> __device__ __forceinline__ uint32_t chunk_offset(int row, int c) {
  return D == 128 ? sw128_offset(row, c) : sw64_offset(row, c);
}

// RL: query rows of a lane, RL * 4 of a group. Columns 2 t, 2 t + 1 of a tile are, in fp32, the
// high and low parts of row 4 x + t (tile x); in bf16 row t and nothing (RL = 1) or rows 2 t, 2 t + 1.
template <typename T, int D, int RL, bool F32>
__global__ void __launch_bounds__(kWarps * 32, 1)
paged_attend_kernel(const AttendParams p, const __grid_constant__ AttendMaps maps) {
  using TL = Tile<D>;
  constexpr int S = TL::kStages, kC = D / 16, kOT = D / 16;   // 16-byte chunks of a row
  constexpr int NT = F32 ? RL : 1;          // column tiles
  extern __shared__ uint8_t smem_raw[];
  __shared__ float4 s_meta[kWarps][kMetaUnits];   // a unit: k_scale, fr 2^13, ev, valid tokens
  __shared__ int s_nan[kWarps][D];          // first token with a NaN value that not all rows see
  __shared__ alignas(8) uint64_t s_bar[kWarps][S];
  __shared__ int s_abort;
  const PagedArgs& a = p.a;
  const lowram_pages& pg = a.pg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int P = pg.page_tokens, upp = P / kUnit;      // 16-token units of a page: 1, 2, 4
  const int lgu = 31 - __clz(upp);
  const int pairs = a.H * p.rp.groups;                // of one sequence
  const int R = a.G * a.n_q;
  const uint32_t ring = ((smem_u32(smem_raw) + 1023u) & ~1023u) + warp * kRingBytes;
  if (threadIdx.x == 0) s_abort = 0;
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(smem_u32(&s_bar[warp][i]), 2);
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
  auto next_seq = [&](int& bb, int& ll, int& nn) {
    do {
      ++bb;
      ll = bb < pg.n_seqs ? paged_len(pg, bb, nullptr) : 0;
      nn = (ll + kStep - 1) / kStep;
    } while (nn == 0 && bb < pg.n_seqs);
  };
  int lb = b, llen = len, lns = ns, lpair = pair, lstep = step, lst = 0, issued = 0;
  int off = 32;                      // the step's first unit among the lanes' page entries
  int uy = -1;                       // this lane's unit: row of its box, -1 for none
  const uint32_t bar0 = smem_u32(&s_bar[warp][0]);
  auto issue = [&]() {
    if (off + 2 > 32) {              // the next 32 units' pages and scales, a lane each
      off = 0;
      const int u = 2 * lstep + lane, h = lpair / p.rp.groups;
      uy = -1;
      float4 me = make_float4(0.f, 0.f, 0.f, 0.f);
      if (u * kUnit < llen) {
        const int page = paged_page(pg, lb, u >> lgu, a.status);
        if (page >= 0) {
          const size_t ph = (size_t)page * a.H + h;
          const float sk = pg.k_scale[ph], sv = pg.v_scale[ph];
          uy = (int)ph * P + (u & (upp - 1)) * kUnit;
          int ev = (int)((__float_as_uint(sv) >> 23) & 255u) - 127;
          ev = min(max(ev, -64), 120);
          me = make_float4(sk, sv * __int_as_float((127 - ev) << 23) * kWeightScale,
                           __int_as_float(ev), __int_as_float(min(llen - u * kUnit, kUnit)));
        }
      }
      s_meta[warp][(2 * issued + lane) & (kMetaUnits - 1)] = me;
    }
    const int mine = lane - off;
    if (mine == 0 || mine == 1) {
      const uint32_t bar = bar0 + 8u * lst;
      const uint32_t dst = ring + lst * TL::kStage + mine * kUnit * D;
      // both units of a step lie in one page of 32 or 64 tokens: one box
      const bool load = uy >= 0 && (mine == 0 || upp == 1);
      mbar_arrive_expect_tx(bar, load ? (upp == 1 ? 2 * kUnit * D : 2 * kStep * D) : 0);
      if (load) {
        tma_load_2d(dst, &maps.k, 0, uy, bar);
        tma_load_2d(dst + TL::kHalf, &maps.v, 0, uy, bar);
      }
    }
    off += 2;
    ++issued;
    if (++lst == S) lst = 0;
    if (++lstep == lns) {
      lstep = 0;
      off = 32;
      if (++lpair == pairs) {
        lpair = 0;
        next_seq(lb, llen, lns);
      }
    }
  };

  // ---- state of the current (sequence, head, group)
  uint32_t qf[NT][kC][2];
  float cs[RL];                     // logit of a row in log2 units per unit of S
  int lim[RL];                      // tokens that the row sees
  float m[RL], l[RL], O[NT][kOT][4];
  // the rows that this lane names to ldmatrix, in a step's K (a unit's) and V
  const int krow = s_token(lane & 15), vrow = v_token(lane & 15) + (lane & 16);
  bool fresh = true, good = true, poison = false;
  int landed = 0, st = 0, row0 = 0, vis = 0;   // vis: tokens that every row of the group sees
  uint32_t parity = 0;
  for (int it = 0; it < n_steps + S; ++it) {
    if (it >= S) {
      if (fresh) {   // the group's queries
        fresh = false;
        const int h = pair / p.rp.groups;
        row0 = (pair - h * p.rp.groups) * p.rp.rows;
        vis = len - a.n_q + row0 / a.G + 1;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          // the row of this lane's column, if it has one
          const int r = F32 ? row0 + 4 * x + (g >> 1) : RL == 1 ? row0 + (g >> 1) : row0 + g;
          const bool has = r < R && (F32 || RL == 2 || (g & 1) == 0);
          float q[kC][4], top = 0.f;
#pragma unroll
          for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) q[c][e] = 0.f;
          if (has) {
            const T* src = (const T*)a.q +
                           (((size_t)b * a.n_q + r / a.G) * a.Hq + h * a.G + r % a.G) * D + 4 * t;
#pragma unroll
            for (int c = 0; c < kC; ++c) VecLoad<T, 4>::load(src + 16 * c, q[c]);
          }
#pragma unroll
          for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(q[c][e]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          int ex = (int)(__float_as_uint(top) >> 23) - 127;
          ex = min(max(ex, -100), 127);
          const float up = __int_as_float((12 - ex + 127) << 23);
#pragma unroll
          for (int c = 0; c < kC; ++c) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              q[c][e] *= up;
              if (F32 && (g & 1)) q[c][e] -= round_f16(q[c][e]);
            }
            qf[x][c][0] = pack_f16x2(q[c][0], q[c][1]);
            qf[x][c][1] = pack_f16x2(q[c][2], q[c][3]);
          }
          const float scale = __int_as_float((ex - 12 + 127) << 23) *
                              (1.4426950408889634f * rsqrtf((float)D));
#pragma unroll
          for (int y = 0; y < RL; ++y)
            if (!F32 || x == y) cs[y] = __shfl_sync(0xffffffffu, scale, 8 * t + (F32 ? 0 : 4 * y));
#pragma unroll
          for (int j = 0; j < kOT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[x][j][e] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < RL; ++x) {
          const int r = row0 + (F32 ? 4 * x + t : RL * t + x);
          lim[x] = r < R ? len - a.n_q + r / a.G + 1 : 0;
          m[x] = -INFINITY;
          l[x] = 0.f;
        }
      }
      good = mbar_wait_bounded(bar0 + 8u * st, parity, abort_flag);
      good = __all_sync(0xffffffffu, good);
      if (!good) break;
      const uint32_t kb = ring + st * TL::kStage, vb = kb + TL::kHalf;
      const float4* meta = &s_meta[warp][(2 * landed) & (kMetaUnits - 1)];   // an even slot
      const float4 me[2] = {meta[0], meta[1]};
      const int valid[2] = {__float_as_int(me[0].w), __float_as_int(me[1].w)};
      ++landed;
      if (++st == S) {
        st = 0;
        parity ^= 1u;
      }
      // S^T = K Q^T: logits in log2 units, masked ones -inf; z[u][x][k]: token row g + 8 k
      float z[2][RL][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float c[2][NT][4];   // even and odd chunks
#pragma unroll
        for (int k = 0; k < kC; k += 2) {
          uint32_t r[4], f[4];
          ldmatrix_x4(kb + u * kUnit * D + chunk_offset<D>(krow, k + (lane >> 4)), r);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            widen(r[2 * y], r[2 * y + 1], f);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              if (k == 0) mma_f16_first(c[y][x], f, qf[x][y][0], qf[x][y][1]);
              else mma_f16(c[y][x], f, qf[x][k + y][0], qf[x][k + y][1]);
            }
          }
        }
#pragma unroll
        for (int x = 0; x < RL; ++x)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int e = 2 * k + (!F32 && RL == 2 ? x : 0), nt = F32 ? x : 0;
            float v = c[0][nt][e] + c[1][nt][e];
            if (F32) v += c[0][nt][2 * k + 1] + c[1][nt][2 * k + 1];
            z[u][x][k] = v * (cs[x] * me[u].x);
          }
      }
      if (valid[0] < kUnit || valid[1] < kUnit || (step + 1) * kStep > vis) {
        // not every token of the step is seen by every row: masked logits, and V rows that are
        // no token (their bytes may be anything) set to zero
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int x = 0; x < RL; ++x)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int tk = s_token(g + 8 * k);
              if (tk >= valid[u] || step * kStep + u * kUnit + tk >= lim[x]) z[u][x][k] = -INFINITY;
            }
          for (int r = 0; r < kUnit; ++r) {
            const int row = u * kUnit + r, tk = step * kStep + row;
            uint8_t* bytes = smem_raw + (vb - smem_u32(smem_raw)) + row * D;
            if (r >= valid[u]) {
              if (lane < D / 4) reinterpret_cast<uint32_t*>(bytes)[lane] = 0;
            } else if (tk >= vis) {
              // a token that only some rows see: its NaN codes would reach the others as 0 * NaN,
              // so they become zeros here and the first of each element is kept for the end
#pragma unroll
              for (int e = lane; e < D; e += 32) {
                const bool nan = (bytes[e] & 127) == 127;
                if (__any_sync(0xffffffffu, nan)) {
                  if (!poison) {
                    poison = true;
                    for (int y = lane; y < D; y += 32) s_nan[warp][y] = 0x7fffffff;
                    __syncwarp();
                  }
                  // the element behind byte e: the chunk's swizzle undone (it is its own inverse)
                  const int el = (int)(chunk_offset<D>(row, e >> 4) - row * D) + (e & 15);
                  if (nan) {
                    s_nan[warp][el] = min(s_nan[warp][el], tk);
                    bytes[e] = 0;
                  }
                }
              }
            }
          }
        }
        __syncwarp();
        fence_proxy_async_smem();   // before a copy fills the stage again
      }
      // reference: max of z + ev
      const float ev[2] = {(float)__float_as_int(me[0].z), (float)__float_as_int(me[1].z)};
      float mn[RL];
      bool grow = false;
#pragma unroll
      for (int x = 0; x < RL; ++x) {
        float v = fmaxf(fmaxf(z[0][x][0], z[0][x][1]) + ev[0], fmaxf(z[1][x][0], z[1][x][1]) + ev[1]);
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        mn[x] = fmaxf(m[x], v);
        grow = grow || mn[x] > m[x];
      }
      if (__any_sync(0xffffffffu, grow)) {
        float corr[RL];
#pragma unroll
        for (int x = 0; x < RL; ++x) {
          corr[x] = mn[x] > m[x] ? ex2_approx(m[x] - mn[x]) : 1.f;
          m[x] = mn[x];
          l[x] *= corr[x];
        }
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int j = 0; j < kOT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[x][j][e] *= corr[F32 ? x : RL == 1 ? 0 : e & 1];
      }
      // weights, as B operands of O^T += V^T P^T
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float back = __int_as_float((127 - __float_as_int(me[u].z)) << 23);   // 2^-ev
        float wgt[RL][2];
#pragma unroll
        for (int x = 0; x < RL; ++x) {
          const float off = m[x] == -INFINITY ? 0.f : ev[u] - m[x];
          const float a0 = ex2_approx(z[u][x][0] + off), a1 = ex2_approx(z[u][x][1] + off);
          l[x] = fmaf(a0 + a1, back, l[x]);
          wgt[x][0] = a0 * me[u].y;
          wgt[x][1] = a1 * me[u].y;
        }
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float hi = wgt[x][k];
            const float lo = F32 ? hi - round_f16(hi) : RL == 2 ? wgt[RL - 1][k] : 0.f;
            pf[u][x][k] = movmatrix_trans(pack_f16x2(hi, lo));
          }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int j = 0; j < kOT; ++j) {
        uint32_t f[4], f0[4], f1[4];
        ldmatrix_b8_trans(vb + chunk_offset<D>(vrow, j), f);   // elements 16 j ..
        widen(f[0], f[1], f0);
        widen(f[2], f[3], f1);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          if (F32) {
            float o[4];
            mma_f16_first(o, f0, pf[0][x][0], pf[0][x][1]);
            mma_f16(o, f1, pf[1][x][0], pf[1][x][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) O[x][j][e] += o[e];
          } else {
            mma_f16(O[x][j], f0, pf[0][x][0], pf[0][x][1]);
            mma_f16(O[x][j], f1, pf[1][x][0], pf[1][x][1]);
          }
        }
      }
      // end of the pair, or of the run: its partial
      const bool last = ++step == ns;
      if (last || landed == n_steps) {
        const size_t slot = (size_t)w + (size_t)b * pairs + pair;
        float* po = p.ws.o + slot * p.rp.rows * D;
        float2* pml = p.ws.ml + slot * p.rp.rows;
#pragma unroll
        for (int x = 0; x < RL; ++x) {
          float v = l[x];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          const int r = F32 ? 4 * x + t : RL * t + x;   // row of the group
          if (row0 + r < R) {
            if (g == 0) pml[r] = make_float2(m[x], v);
#pragma unroll
            for (int j = 0; j < kOT; ++j)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int el = 16 * j + g + 8 * k;
                float o = F32 ? O[F32 ? x : 0][j][2 * k] + O[F32 ? x : 0][j][2 * k + 1]
                              : O[0][j][2 * k + (RL == 2 ? x : 0)];
                if (poison && s_nan[warp][el] < lim[x]) o = __int_as_float(0x7fffffff);
                po[(size_t)r * D + el] = o;
              }
          }
        }
        fresh = true;
        poison = false;
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
    if (it < n_steps) issue();
  }
  if (!good) {   // a wait gave up: the copies still in flight land first
    if (lane == 0) raise_status(a.status, kStatusTimeout);
    for (; landed < issued; ++landed) {
      int dummy = 0;
      mbar_wait_bounded(bar0 + 8u * st, parity, &dummy);
      if (++st == S) {
        st = 0;
        parity ^= 1u;
      }
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
    if constexpr (E == 4) {
      const float4 y = *reinterpret_cast<const float4*>(po + s * so);
      o[0] = y.x; o[1] = y.y; o[2] = y.z; o[3] = y.w;
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

template <typename T, int D, int RL, bool F32>
cudaError_t attend_t(const AttendParams& p, int num_sms, cudaStream_t s) {
  const PagedArgs& a = p.a;
  AttendMaps maps;
  const uint64_t rows = (uint64_t)a.pg.n_pages * a.H * a.pg.page_tokens;
  const uint32_t box = a.pg.page_tokens < kStep ? kUnit : kStep;
  if (!make_tensor_map_2d(&maps.k, a.pg.k_code, kMapBytes, D, rows, D, box, D, 256) ||
      !make_tensor_map_2d(&maps.v, a.pg.v_code, kMapBytes, D, rows, D, box, D, 256))
    return cudaErrorInvalidValue;
  const size_t smem = (size_t)kWarps * kRingBytes + 1024;
  auto kern = paged_attend_kernel<T, D, RL, F32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<num_sms < kMaxCtas ? num_sms : kMaxCtas, kWarps * 32, smem, s>>>(p, maps);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  paged_combine_kernel<T, D><<<dim3(a.n_q * a.Hq, a.pg.n_seqs), kCombineThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int D, bool F32>
cudaError_t attend_d(const AttendParams& p, int num_sms, cudaStream_t s) {
  return p.rp.rows == 4 ? attend_t<T, D, 1, F32>(p, num_sms, s)
                        : attend_t<T, D, 2, F32>(p, num_sms, s);
}

}  // namespace

size_t paged_attend_workspace_bytes(int H, int G, int d, int n_seqs, int n_q) {
  size_t total = 0;
  ws_layout(nullptr, H, row_plan(G, n_q), d, n_seqs, &total);
  return total;
}

cudaError_t launch_paged_attend(const PagedArgs& a, int num_sms, cudaStream_t s) {
  AttendParams p{};
  p.a = a;
  p.rp = row_plan(a.G, a.n_q);
  p.ws = ws_layout(a.ws, a.H, p.rp, a.d, a.pg.n_seqs, nullptr);
  if (a.dtype == LOWRAM_DTYPE_BF16)
    return a.d == 128 ? attend_d<__nv_bfloat16, 128, false>(p, num_sms, s)
                      : attend_d<__nv_bfloat16, 64, false>(p, num_sms, s);
  return a.d == 128 ? attend_d<float, 128, true>(p, num_sms, s)
                    : attend_d<float, 64, true>(p, num_sms, s);
}

}  // namespace lowram
