// Attention over the paged 8-bit cache for the last n_q tokens of every sequence:
//   z_t = (q . k_code_t) k_scale / sqrt(d),  out = sum_t softmax(z)_t v_code_t v_scale.
//
// Bound by bytes: each group of 16 query rows of a head (8 in fp32) reads each code once
// (2 sum(len) H d bytes a group), for 4 G n_q operations a pair of codes; with several groups,
// and in fp32, by instructions. The work is cut into steps of 8 KB (32 tokens, 64 for d = 64) of one (sequence, KV
// head, group of query rows), all in one list, an equal run of them for every warp of the GPU, so
// ragged batches and single long sequences fill it alike. A warp streams its run alone: it issues
// TMA boxes into its own ring of stages, holds the queries as matrix fragments in registers, and
// writes one partial (reference, sum, output) for every (sequence, head, group) that its run
// touches. A second kernel merges the partials of a row.
//
// Two stages a warp, not three: with 192 KB of an SM always asked for, four groups of ten SMs get
// a tenth less of the bandwidth than the others and end that much later (batch 8 at 128K tokens:
// SMs end at 280 .. 350 us); with 128 KB all get the same (300 .. 319 us; the call 354 -> 326 us;
// now, over caches that find nothing in the L2, 318 .. 345 by GPU, 6.2 .. 6.7 TB/s).
// Handing the list's end out in short runs instead cost more than it evened out (a run's queries,
// partial and pages are about 3 us of a warp).
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
// the softmax's reference and sum and the output are fp32. A weight a = 2^(z - m + 8) is rounded
// to fp16: in two columns where they are free (fp32, and up to 4 bf16 rows: 2^-22), in one for
// more bf16 rows (2^-11, eight times finer than the output; a second column would double their
// products, and they are bound by instructions). The row's reference m is the largest z so far to
// within 2^6, so a <= 2^14.
// The matrix unit cuts its sums toward zero, by 2^-24 of the sum each time, so a step's product
// starts from zero and is added to the output in fp32: carried on in the unit, 2^21 tokens of a
// run came out 1.3 % too small.
// Values' scales. A step's product is added times 2^(e - 40), e the largest exponent of the
// step's v_scales; a weight carries what its page's scale is below that (>= 2^-8, or the next
// form is taken), and the output is held in units of 2^32, where every sum of admitted scales
// (2^-64 .. 2^120) is a normal number. So scales reach neither the softmax's sum nor one
// another's digits. Where a unit's scale is more than 2^8 above the least of the run, its values
// may matter at weights that fp16 cannot hold beside 1: the units of such a step each take their
// own largest z as reference, and what that is above or below m goes into the fp32 factor.
// (Every third page 2^20 smaller: batch 8 to 64K tokens 101.0 -> 102.3 us, fp32 40K 40.1 -> 46.5,
// 5 drafted tokens 45.0 -> 54.1; near scales pay two integer operations a unit for the choice.)
#include <cuda.h>

#include "paged_common.cuh"
#include "sm100_ptx.cuh"

namespace lowram {
namespace {

using namespace sm100;

constexpr int kWarps = 8;
constexpr int kUnit = 16;                 // tokens of a matrix tile
constexpr int kMetaUnits = 64;            // a warp's ring of units' scales
constexpr int kMaxCtas = 160;             // bound of the workspace; the grid is one CTA an SM
constexpr int kStages = 2;                // a warp's ring: 16 KB
constexpr uint32_t kHalfBytes = 4096;     // K (or V) of a step
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr uint32_t kRingBytes = kStages * kStageBytes;
constexpr int kWeightExp = 8;             // weights times 2^8: in fp16 normal down to 2^-22
constexpr float kWeightScale = 1 << kWeightExp;
constexpr int kOutExp = 32;               // the output's unit 2^32, with the weights' 2^8 taken out
constexpr int kLeastExp = -64;            // of a scale
constexpr int kNearExp = 8;               // spread of scales that weights may carry
constexpr float kSlack = 6.f;             // log2 of what a weight may exceed its reference by
constexpr int kCombineThreads = 256;

template <int D> struct Tile {
  static constexpr int kStep = kHalfBytes / D;       // tokens of a step: 32 (d = 128), 64
  static constexpr int kUnits = kStep / kUnit;       // 2, 4
};

struct AttendMaps {
  CUtensorMap k;   // [n_pages * H * page_tokens rows][d] bytes, box d x min(page_tokens, step),
                   // swizzled by d bytes
  CUtensorMap v;
};

// Query rows of one (sequence, KV head): r = j G + g, in groups of `rows`.
struct RowPlan {
  int rows, groups;   // rows of a group (4, 8; bf16: 16), groups
};
inline RowPlan row_plan(int G, int n_q, int dtype) {
  const int R = G * n_q;
  RowPlan p;
  p.rows = R <= 4 ? 4 : R <= 8 || dtype != LOWRAM_DTYPE_BF16 ? 8 : 16;
  p.groups = (R + p.rows - 1) / p.rows;
  return p;
}

// Workspace: first step of every sequence (of one pair each) and their total, for the merge of
// more than 32 sequences; the partials' (m, l) and outputs. The partial of warp w for pair x
// (= (b H + h) groups + group) is number w + x: both only grow along the list of steps.
struct AttendWs {
  long long* first;   // [n_seqs + 1]
  float2* ml;   // [slots][rows]
  float* o;     // [slots][rows][d]
};
inline size_t ws_align(size_t x) { return (x + 255) / 256 * 256; }
inline AttendWs ws_layout(void* ws, int H, const RowPlan& rp, int d, int n_seqs, size_t* total) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  const size_t slots = (size_t)kMaxCtas * kWarps + (size_t)n_seqs * H * rp.groups;
  AttendWs w;
  w.first = reinterpret_cast<long long*>(p);
  size_t o = ws_align((size_t)(n_seqs + 1) * sizeof(long long));
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
  int n_warps;   // of the attend kernel
};

// x / y for y > 0, x >= 0: by 32 bits where they do (a 64-bit division is a tenth of a
// microsecond, which the shortest calls see).
__device__ __forceinline__ long long div_pos(long long x, int y) {
  return x <= 0x7fffffffLL ? (long long)((unsigned)x / (unsigned)y) : x / y;
}
// Steps of a warp's run, of `total` in the list: below 2^31 (n_seqs, pairs and lengths bound it).
__device__ __forceinline__ int run_steps(long long total, int n_warps) {
  return total > 0 ? (int)div_pos(total + n_warps - 1, n_warps) : 1;
}

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
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }
// Over the lanes of a fragment's column.
__device__ __forceinline__ float lanes_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
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

// RL: query rows of a lane, 4 RL of a group. Columns 2 t, 2 t + 1 of a tile are, in fp32, the
// high and low parts of row 4 x + t (tile x); in bf16 row t, its weights in two parts and its
// query in one (RL = 1), or rows 8 x + 2 t, 8 x + 2 t + 1 (tile x).
//
// 208 registers where RL = 1: a CTA of the merge then fits beside one of this kernel and is set up
// early (with 211: one 4K sequence 15.0 us instead of 9.7).
template <typename T, int D, int RL, bool F32>
__global__ void __maxnreg__(RL == 1 ? 208 : 255)
paged_attend_kernel(const AttendParams p, const __grid_constant__ AttendMaps maps) {
  using TL = Tile<D>;
  constexpr int S = kStages, U = TL::kUnits, kStep = TL::kStep;
  constexpr int kC = D / 16, kOT = D / 16;          // 16-byte chunks of a row
  constexpr int NT = F32 ? RL : (RL + 1) / 2;       // column tiles
  constexpr bool kParts = F32 || RL == 1;           // weights in two columns
  extern __shared__ uint8_t smem_raw[];
  __shared__ float4 s_meta[kWarps][kMetaUnits];   // a unit: k_scale, v_scale, its exponent, tokens
  __shared__ int4 s_desc[kWarps][S];        // a stage's step: sequence, pair, first token, length
  __shared__ int2 s_part[kWarps][S];        // its partial; 1: begins one, 2: ends it
  __shared__ int s_nan[kWarps][D];          // first token with a NaN value that not all rows see
  __shared__ alignas(8) uint64_t s_bar[kWarps][S];
  __shared__ int s_abort;
  const PagedArgs& a = p.a;
  const lowram_pages& pg = a.pg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int P = pg.page_tokens, lgu = 31 - __clz(P / kUnit);   // log2 units of a page: 0, 1, 2
  const int pairs = a.H * p.rp.groups;                // of one sequence
  const int R = a.G * a.n_q;
  const uint32_t ring = ((smem_u32(smem_raw) + 1023u) & ~1023u) + warp * kRingBytes;
  if (threadIdx.x == 0) s_abort = 0;
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(smem_u32(&s_bar[warp][i]), U);
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  // only now: the merge reads the lengths before its own wait, so what wrote them must have ended
  grid_launch_dependents();
  volatile int* abort_flag = &s_abort;

  // ---- the list of steps
  auto steps_of = [&](int n) { return (n + kStep - 1) / kStep; };
  auto scan = [&](int x) {   // inclusive, over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  const int len0 = lane < pg.n_seqs ? paged_len(pg, lane, a.status) : 0;
  auto len_at = [&](int b) {   // b = lane + 32 i
    return b < 32 ? len0 : b < pg.n_seqs ? paged_len(pg, b, nullptr) : 0;
  };
  long long total = 0;
  for (int b0 = 0; b0 < pg.n_seqs; b0 += 32) {
    const int b = b0 + lane;
    const int n = b < 32 ? len0 : b < pg.n_seqs ? paged_len(pg, b, a.status) : 0;
    total += __reduce_add_sync(0xffffffffu, steps_of(n));
  }
  if (pg.n_seqs > 32 && warp == 0 && blockIdx.x == 0) {   // for the merge
    long long at = 0;
    for (int b0 = 0; b0 < pg.n_seqs; b0 += 32) {
      const int n = steps_of(len_at(b0 + lane)), x = scan(n);
      if (b0 + lane < pg.n_seqs) p.ws.first[b0 + lane] = at + x - n;
      at += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) p.ws.first[pg.n_seqs] = total;
  }
  total *= pairs;
  // consecutive runs go to different SMs, so that little work still uses many of them
  const int run = warp * gridDim.x + blockIdx.x;

  // ---- the loader. It works in batches of up to 32 units (a lane each) of one pair, and looks
  // up a batch's pages, then its scales, while the batch before is being issued.
  constexpr int kBatch = 32 / U;     // steps of a batch
  const uint32_t bar0 = smem_u32(&s_bar[warp][0]);
  int lb = 0, llen = 0, lns = 1, lpair = 0, lstep = 0;   // cursor: behind the batch looked up last
  int left = 0, flag = 1;            // steps left of the run; the next batch begins a partial
  int nb = 0, npair = 0, ntok = 0, nlen = 0, ncnt = 0, nslot = 0, nflag = 0;   // next batch
  int npage = -1, nvalid = 0;        // its unit of this lane: page, tokens, scales
  float nsk = 0.f, nsv = 0.f;
  bool nscaled = false;
  int cb = 0, cpair = 0, ctok = 0, clen = 0, ccnt = 0, cslot = 0, cflag = 0;   // current batch
  int uy = -1, off = 0;              // its unit of this lane: row of its box; the step's first unit
  int lst = 0, issued = 0;
  {   // where the run begins: sequence, pair, step
    const int steps = run_steps(total, p.n_warps);
    const long long r0 = min(total, (long long)run * steps);
    left = (int)(min(total, r0 + steps) - r0);
    long long at = 0;
    for (int b0 = 0; left > 0 && b0 < pg.n_seqs; b0 += 32) {
      const int n = len_at(b0 + lane), x = scan(steps_of(n));
      const unsigned past = __ballot_sync(0xffffffffu, (at + x) * pairs > r0);
      if (past) {
        const int src = __ffs(past) - 1;
        lb = b0 + src;
        llen = __shfl_sync(0xffffffffu, n, src);
        lns = steps_of(llen);
        const long long in = r0 - (at + __shfl_sync(0xffffffffu, x, src) - lns) * pairs;
        lpair = (int)div_pos(in, lns);
        lstep = (int)(in - (long long)lpair * lns);
        break;
      }
      at += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  auto look_up = [&]() {             // the next batch: where it lies, and its pages
    ncnt = 0;
    if (left == 0) return;
    nb = lb;
    npair = lpair;
    ntok = lstep * kStep;
    nlen = llen;
    ncnt = min(min(kBatch, lns - lstep), left);
    nslot = run + lb * pairs + lpair;
    const int u = U * lstep + lane;
    nvalid = min(max(llen - u * kUnit, 0), kUnit);
    if (lane >= U * ncnt) nvalid = 0;
    npage = nvalid > 0 ? pg.table[(size_t)lb * pg.max_pages + (u >> lgu)] : -1;
    nscaled = false;
    lstep += ncnt;
    left -= ncnt;
    const bool ends = lstep == lns || left == 0;
    nflag = flag | (ends ? 2 : 0);
    flag = ends ? 1 : 0;
    if (lstep == lns && left > 0) {
      lstep = 0;
      if (++lpair == pairs) {
        lpair = 0;
        do {
          ++lb;
          llen = lb >= pg.n_seqs ? 0 : lb < 32 ? __shfl_sync(0xffffffffu, len0, lb)
                                               : paged_len(pg, lb, nullptr);
          lns = steps_of(llen);
        } while (lns == 0 && lb < pg.n_seqs);
      }
    }
  };
  auto look_up_scales = [&]() {
    nscaled = true;
    if (nvalid > 0 && (npage < 0 || npage >= pg.n_pages)) {
      raise_status(a.status, kStatusDeviceCheck);
      nvalid = 0;
    }
    nsk = nsv = 0.f;   // no unit: a stale scale, were it NaN, would reach masked weights as 0 * NaN
    if (nvalid > 0) {
      const size_t ph = (size_t)npage * a.H + npair / p.rp.groups;
      nsk = pg.k_scale[ph];
      nsv = pg.v_scale[ph];
    }
  };
  auto issue = [&]() {
    const bool first = ccnt == 0;
    if (first) {                     // the next batch becomes the current one
      if (!nscaled) look_up_scales();
      cb = nb; cpair = npair; ctok = ntok; clen = nlen; ccnt = ncnt; cslot = nslot; cflag = nflag;
      const int h = cpair / p.rp.groups;
      const int u = ctok / kUnit + lane;
      uy = nvalid > 0 ? (npage * a.H + h) * P + (u & ((1 << lgu) - 1)) * kUnit : -1;
      off = 0;
    } else if (!nscaled) {
      look_up_scales();
    }
    const int mine = lane - off;
    if (mine >= 0 && mine < U) {
      const uint32_t bar = bar0 + 8u * lst;
      const uint32_t dst = ring + lst * kStageBytes + mine * kUnit * D;
      // units of one page (and step) come as one box
      const bool load = uy >= 0 && (mine & ((1 << lgu) - 1)) == 0;
      mbar_arrive_expect_tx(bar, load ? 2 * min(P, kStep) * D : 0);
      if (load) {
        tma_load_2d(dst, &maps.k, 0, uy, bar);
        tma_load_2d(dst + kHalfBytes, &maps.v, 0, uy, bar);
      }
    }
    if (first) {                     // behind the copies: the scales may still be on their way
      int ev = (int)((__float_as_uint(nsv) >> 23) & 255u) - 127;
      ev = nvalid > 0 ? min(max(ev, kLeastExp), 120) : kLeastExp - 1;   // below all: no unit
      s_meta[warp][(U * issued + lane) & (kMetaUnits - 1)] =
          make_float4(nsk, nsv, __int_as_float(ev), __int_as_float(nvalid));
      look_up();
    }
    --ccnt;
    if (lane == 0) {
      s_desc[warp][lst] = make_int4(cb, cpair, ctok, clen);
      s_part[warp][lst] = make_int2(cslot, ccnt == 0 ? cflag : cflag & 1);
    }
    cflag &= 2;                      // only the batch's first step begins a partial
    ctok += kStep;
    off += U;
    ++issued;
    if (++lst == S) lst = 0;
    __syncwarp();
  };
  look_up();

  // ---- state of the current (sequence, head, group)
  auto row_of = [&](int x) {        // this lane's x-th row of the group
    return F32 ? 4 * x + t : RL == 1 ? t : 8 * (x >> 1) + 2 * t + (x & 1);
  };
  uint32_t qf[NT][kC][2];
  float cs[RL];                     // logit of a row in log2 units per unit of S
  int lim[RL];                      // tokens that the row sees
  float m[RL], l[RL], O[NT][kOT][4];
  unsigned least_ev = 0;            // least exponent of a value's scale so far, from kLeastExp
  // the rows that this lane names to ldmatrix, in a step's K (a unit's) and V
  const int krow = s_token(lane & 15), vrow = v_token(lane & 15) + (lane & 16);   // two units' V
  bool good = true, poison = false;
  int landed = 0, st = 0, row0 = 0, vis = 0;   // vis: tokens that every row of the group sees
  uint32_t parity = 0;
  for (;;) {
    if (ccnt + ncnt > 0 && issued < landed + S) {
      __syncwarp();   // every lane has read the stage (and its meta) that is filled again
      issue();
      if (ccnt + ncnt > 0 && issued < landed + S) continue;
    }
    if (landed == issued) break;
    {
      const int4 ds = s_desc[warp][st];   // sequence, pair, first token, length
      const int2 part = s_part[warp][st];
      const int tok0 = ds.z;
      if (part.y & 1) {   // a new (sequence, head, group): its queries
        const int b = ds.x, h = ds.y / p.rp.groups, len = ds.w;
        poison = false;
        least_ev = 0xffffu;
        row0 = (ds.y - h * p.rp.groups) * p.rp.rows;
        vis = len - a.n_q + row0 / a.G + 1;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          // the row of this lane's column, if it has one
          const int r = row0 + (F32 ? 4 * x + (g >> 1) : RL == 1 ? g >> 1 : 8 * x + g);
          const bool has = r < R && (F32 || RL > 1 || (g & 1) == 0);
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
            if (x == (F32 ? y : y >> 1))
              cs[y] = __shfl_sync(0xffffffffu, scale, 8 * t + (F32 ? 0 : 4 * (y & 1)));
#pragma unroll
          for (int j = 0; j < kOT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[x][j][e] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < RL; ++x) {
          const int r = row0 + row_of(x);
          lim[x] = r < R ? len - a.n_q + r / a.G + 1 : 0;
          m[x] = -INFINITY;
          l[x] = 0.f;
        }
      }
      good = mbar_wait_bounded(bar0 + 8u * st, parity, abort_flag);
      good = __all_sync(0xffffffffu, good);
      if (!good) break;
      const uint32_t kb = ring + st * kStageBytes, vb = kb + kHalfBytes;
      const float4* meta = &s_meta[warp][(U * landed) & (kMetaUnits - 1)];   // a multiple of U
      ++landed;
      if (++st == S) {
        st = 0;
        parity ^= 1u;
      }
      // S^T = K Q^T: logits in log2 units, masked ones -inf; z[u][x][k]: token row g + 8 k
      float z[U][RL][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float c[2][NT][4];   // even and odd chunks
        const float sk = meta[u].x;
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
            const int e = 2 * k + (F32 ? 0 : x & 1), nt = F32 ? x : x >> 1;
            float v = c[0][nt][e] + c[1][nt][e];
            if (F32) v += c[0][nt][2 * k + 1] + c[1][nt][2 * k + 1];
            z[u][x][k] = v * (cs[x] * sk);
          }
      }
      int least = kUnit;
#pragma unroll
      for (int u = 0; u < U; ++u) least = min(least, __float_as_int(meta[u].w));
      if (least < kUnit || tok0 + kStep > vis) {
        // not every token of the step is seen by every row: masked logits, and V rows that are
        // no token (their bytes may be anything) set to zero
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int valid = __float_as_int(meta[u].w);
#pragma unroll
          for (int x = 0; x < RL; ++x)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int tk = s_token(g + 8 * k);
              if (tk >= valid || tok0 + u * kUnit + tk >= lim[x]) z[u][x][k] = -INFINITY;
            }
          // rows from `valid` on lie together
          for (uint32_t o = (u * kUnit + valid) * D + 16 * lane; o < (u + 1) * kUnit * D; o += 512)
            st_shared_v4(vb + o, 0, 0, 0, 0);
          // Tokens that only some rows see: their NaN codes would reach the others as 0 * NaN, so
          // they become zeros here and the first of each element is kept for the end.
          for (int row = max(vis - tok0, u * kUnit); row < u * kUnit + valid; ++row) {
            uint8_t* bytes = smem_raw + (vb - smem_u32(smem_raw)) + row * D;
#pragma unroll
            for (int e = lane; e < D; e += 32) {
              const bool nan = (bytes[e] & 127) == 127;
              if (__any_sync(0xffffffffu, nan)) {
                if (!poison) {
                  poison = true;
                  __syncwarp();   // the pair before has read its entries
                  for (int y = lane; y < D; y += 32) s_nan[warp][y] = 0x7fffffff;
                  __syncwarp();
                }
                // the element behind byte e: the chunk's swizzle undone (it is its own inverse)
                const int el = (int)(chunk_offset<D>(row, e >> 4) - row * D) + (e & 15);
                if (nan) {
                  s_nan[warp][el] = min(s_nan[warp][el], tok0 + row);
                  bytes[e] = 0;
                }
                __syncwarp();   // another lane holds this element in the next row
              }
            }
          }
        }
        __syncwarp();
        fence_proxy_async_smem();   // before a copy fills the stage again
      }
      // reference: the max of z, moved only when a token exceeds it by 2^kSlack: few steps then
      // pay for the reduction over the lanes and the output's rescaling
      float mn[RL];
      bool grow = false;
#pragma unroll
      for (int x = 0; x < RL; ++x) {
        mn[x] = fmaxf(z[0][x][0], z[0][x][1]);
#pragma unroll
        for (int u = 1; u < U; ++u) mn[x] = fmaxf(mn[x], fmaxf(z[u][x][0], z[u][x][1]));
        grow = grow || mn[x] > m[x] + kSlack;
      }
      if (__any_sync(0xffffffffu, grow)) {
        float corr[RL];   // the factor's square root: tiny weights of huge values are no zeros
#pragma unroll
        for (int x = 0; x < RL; ++x) {
          const float v = lanes_max(mn[x]);
          corr[x] = v > m[x] ? ex2_approx(0.5f * (m[x] - v)) : 1.f;
          m[x] = fmaxf(m[x], v);
          l[x] *= corr[x] * corr[x];
        }
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int j = 0; j < kOT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float c = corr[kParts ? x : 2 * x + (e & 1)];
              O[x][j][e] = O[x][j][e] * c * c;
            }
      }
      // weights, as B operands of O^T += V^T P^T
      uint32_t pf[U][NT][2];
      auto operand = [&](const float (&wgt)[RL][2], uint32_t (&f)[NT][2]) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float hi = wgt[kParts ? x : 2 * x][k];
            const float lo = kParts ? hi - round_f16(hi) : wgt[kParts ? 0 : 2 * x + 1][k];
            f[x][k] = movmatrix_trans(pack_f16x2(hi, lo));
          }
      };
      int top = kLeastExp - 1;   // the step's largest exponent of a value's scale
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int ev = __float_as_int(meta[u].z);
        top = max(top, ev);
        least_ev = min(least_ev, (unsigned)(ev - kLeastExp));   // no unit: above all
      }
      if (top - kLeastExp <= (int)least_ev + kNearExp) {
        const float down = pow2f(-top);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float sv = meta[u].y * down;
          float wgt[RL][2];
#pragma unroll
          for (int x = 0; x < RL; ++x) {
            const float off = m[x] == -INFINITY ? 0.f : kWeightExp - m[x];
            const float a0 = ex2_approx(z[u][x][0] + off), a1 = ex2_approx(z[u][x][1] + off);
            l[x] += a0 + a1;
            wgt[x][0] = a0 * sv;
            wgt[x][1] = a1 * sv;
          }
          operand(wgt, pf[u]);
        }
        // O^T += V^T P^T
        const float unit = pow2f(top - kWeightExp - kOutExp);
#pragma unroll
        for (int j = 0; j < kOT; ++j) {
          float o[NT][4];
#pragma unroll
          for (int u = 0; u < U; u += 2) {
            uint32_t f[4], f0[4], f1[4];
            ldmatrix_b8_trans(vb + chunk_offset<D>(u * kUnit + vrow, j), f);   // elements 16 j ..
            widen(f[0], f[1], f0);
            widen(f[2], f[3], f1);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              if (u == 0) mma_f16_first(o[x], f0, pf[u][x][0], pf[u][x][1]);
              else mma_f16(o[x], f0, pf[u][x][0], pf[u][x][1]);
              mma_f16(o[x], f1, pf[u + 1][x][0], pf[u + 1][x][1]);
            }
          }
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[x][j][e] = fmaf(o[x][e], unit, O[x][j][e]);
        }
      } else {
        // scales far apart: a unit at a time, from its own largest z. Four units are not unrolled
        // (unit 0 of z, the others moved up): they would not fit the registers.
        constexpr bool kRoll = U > 2;
#pragma unroll (kRoll ? 1 : U)
        for (int u = 0; u < U; ++u) {
          const int zu = kRoll ? 0 : u;
          const int ev = __float_as_int(meta[u].z);
          const float sv = meta[u].y * pow2f(-ev);
          float wgt[RL][2], unit[RL];
#pragma unroll
          for (int x = 0; x < RL; ++x) {
            const float r = lanes_max(fmaxf(z[zu][x][0], z[zu][x][1]));
            const bool some = r != -INFINITY;
            const float off = some ? kWeightExp - r : 0.f;
            const float back = some ? exp2f(r - m[x]) : 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              wgt[x][k] = ex2_approx(z[zu][x][k] + off);
              l[x] = fmaf(wgt[x][k], back, l[x]);
              if (kRoll) {
#pragma unroll
                for (int w = 1; w < U; ++w) z[w - 1][x][k] = z[w][x][k];
              }
            }
            unit[x] = some ? exp2f(r - m[x] + (float)(ev - kWeightExp - kOutExp)) * sv : 0.f;
          }
          operand(wgt, pf[zu]);
#pragma unroll
          for (int j = 0; j < kOT; ++j) {
            uint32_t f[4], fu[4];
            ldmatrix_b8_trans(vb + chunk_offset<D>((u & ~1) * kUnit + vrow, j), f);
            widen(u & 1 ? f[2] : f[0], u & 1 ? f[3] : f[1], fu);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              float o[4];
              mma_f16_first(o, fu, pf[zu][x][0], pf[zu][x][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                O[x][j][e] = fmaf(o[e], unit[kParts ? x : 2 * x + (e & 1)], O[x][j][e]);
            }
          }
        }
      }
      // end of the pair, or of the run: its partial
      if (part.y & 2) {
        float* po = p.ws.o + (size_t)part.x * p.rp.rows * D;
        float2* pml = p.ws.ml + (size_t)part.x * p.rp.rows;
#pragma unroll
        for (int x = 0; x < RL; ++x) {
          float v = l[x];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          const int r = row_of(x);
          if (row0 + r < R) {
            if (g == 0) pml[r] = make_float2(m[x], v);
#pragma unroll
            for (int j = 0; j < kOT; ++j)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int el = 16 * j + g + 8 * k;
                float o = kParts ? O[kParts ? x : 0][j][2 * k] + O[kParts ? x : 0][j][2 * k + 1]
                                 : O[x >> 1][j][2 * k + (x & 1)];
                if (poison && s_nan[warp][el] < lim[x]) o = __int_as_float(0x7fffffff);
                po[(size_t)r * D + el] = o;
              }
          }
        }
      }
    }
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

// Weight 2^(m - top) of a partial with reference m: 1 where it saw nothing and holds zeros (a NaN
// sum must stay one).
__device__ __forceinline__ float weight_of(float m, float top) {
  return m == -INFINITY ? 1.f : ex2_approx(m - top);
}
// Its root, to be applied twice: a weight that is no fp32 number may be that of huge values.
__device__ __forceinline__ float root_weight(float m, float top) {
  return weight_of(0.5f * m, 0.5f * top);
}
__device__ __forceinline__ bool is_tiny(float m, float top) {
  return m != -INFINITY && m - top < -126.f;
}

// One CTA a query row: out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s over the partials
// of its pair. The warps take every eighth partial, four of them in flight together (one after
// another, the 129 partials of a 4K sequence took 6 us). Where the partials lie follows from the
// lengths; up to 32 sequences it is worked out while the first kernel runs. A compressed prefix
// joins as one more partial. Five CTAs an SM, so 48 registers: one then fits beside a CTA of the
// first kernel (with 66: one sequence of 600 tokens 7.4 us instead of 6.7).
template <typename T, int D>
__global__ void __launch_bounds__(kCombineThreads, 5) paged_combine_kernel(const AttendParams p) {
  constexpr int E = D / 32, kW = kCombineThreads / 32, kStep = Tile<D>::kStep;
  const PagedArgs& a = p.a;
  const lowram_pages& pg = a.pg;
  const int hq = blockIdx.x % a.Hq, j = blockIdx.x / a.Hq, b = blockIdx.y;
  const int h = hq / a.G, r = j * a.G + hq % a.G;
  const int grp = r / p.rp.rows, rg = r % p.rp.rows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = a.H * p.rp.groups, pair = h * p.rp.groups + grp;
  long long total, before;
  int ns;
  if (pg.n_seqs <= 32) {
    const int n = lane < pg.n_seqs ? (paged_len(pg, lane, nullptr) + kStep - 1) / kStep : 0;
    total = __reduce_add_sync(0xffffffffu, n);
    before = __reduce_add_sync(0xffffffffu, lane < b ? n : 0);
    ns = __shfl_sync(0xffffffffu, n, b);
  } else {
    grid_dependency_wait();
    total = p.ws.first[pg.n_seqs];
    before = p.ws.first[b];
    ns = (int)(p.ws.first[b + 1] - before);
  }
  const int share = run_steps(total * pairs, p.n_warps);
  const long long step0 = before * pairs + (long long)pair * ns;
  const int first = (int)div_pos(step0, share);
  const int count = ns > 0 ? (int)div_pos(step0 + ns - 1, share) - first + 1 : 0;
  const size_t slot0 = (size_t)first + (size_t)b * pairs + pair;
  const float2* ml = p.ws.ml + slot0 * p.rp.rows + rg;
  const float* po = p.ws.o + (slot0 * p.rp.rows + rg) * D + lane * E;
  const size_t so = (size_t)p.rp.rows * D;
  const size_t row = ((size_t)b * a.n_q + j) * a.Hq + hq;
  grid_dependency_wait();
  grid_launch_dependents();
  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  bool tiny = false;
  constexpr int kU = 4;   // partials of a warp in flight together
  for (int s0 = warp; s0 < count; s0 += kU * kW) {
    float2 x[kU];
    float o[kU][E], mn = m;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int s = s0 + u * kW;
      x[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) o[u][e] = 0.f;
      if (s < count) {
        x[u] = ml[(size_t)s * p.rp.rows];
        if constexpr (E == 4) {
          const float4 y = *reinterpret_cast<const float4*>(po + s * so);
          o[u][0] = y.x; o[u][1] = y.y; o[u][2] = y.z; o[u][3] = y.w;
        } else {
          const float2 y = *reinterpret_cast<const float2*>(po + s * so);
          o[u][0] = y.x; o[u][1] = y.y;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) mn = fmaxf(mn, x[u].x);
    tiny = tiny || is_tiny(m, mn);
#pragma unroll
    for (int u = 0; u < kU; ++u) tiny = tiny || is_tiny(x[u].x, mn);
    const float c = weight_of(m, mn);
    m = mn;
    l *= c;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= c;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const float w = weight_of(x[u].x, mn);
      l = fmaf(w, x[u].y, l);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, o[u][e], acc[e]);
    }
  }
  if (tiny) {   // (rare) once more, from the largest reference and in two steps
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int s = warp; s < count; s += kW) {
      const float2 x = ml[(size_t)s * p.rp.rows];
      const float w = root_weight(x.x, m);
      l = fmaf(w * w, x.y, l);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, po[s * so + e] * w, acc[e]);
    }
  }
  __shared__ float s_m[kW], s_l[kW], s_o[kW][D];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f, w[kW];
#pragma unroll
  for (int x = 0; x < kW; ++x) M = fmaxf(M, s_m[x]);
  float pw = 0.f, pl = 0.f;   // a compressed prefix's softmax, max in log2 units
  if (a.pre_ml) {
    const float pm = a.pre_ml[2 * row] * 1.4426950408889634f;
    M = fmaxf(M, pm);
    pw = root_weight(pm, M);
    pl = a.pre_ml[2 * row + 1] * kWeightScale;
    L = pl * pw * pw;
  }
#pragma unroll
  for (int x = 0; x < kW; ++x) {
    w[x] = root_weight(s_m[x], M);
    L = fmaf(w[x] * w[x], s_l[x], L);
  }
  const float inv = L == 0.f ? 0.f : pow2f(kWeightExp + kOutExp) / L;
  if (threadIdx.x < D) {
    float o = 0.f;
#pragma unroll
    for (int x = 0; x < kW; ++x) o = fmaf(w[x], s_o[x][threadIdx.x] * w[x], o);
    if (a.pre_ml)
      o = fmaf(pw, a.pre_out[row * D + threadIdx.x] * pow2f(-kWeightExp - kOutExp) * pl * pw, o);
    ((T*)a.out)[row * D + threadIdx.x] = from_f<T>(o * inv);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[row] = L == 0.f ? -INFINITY : fmaf(M, 0.69314718055994531f, logf(L * (1.f / kWeightScale)));
}

template <typename T, int D, int RL, bool F32>
cudaError_t attend_t(const AttendParams& p, cudaStream_t s) {
  const PagedArgs& a = p.a;
  AttendMaps maps;
  const uint64_t rows = (uint64_t)a.pg.n_pages * a.H * a.pg.page_tokens;
  const uint32_t box = a.pg.page_tokens < Tile<D>::kStep ? a.pg.page_tokens : Tile<D>::kStep;
  if (!make_tensor_map_2d(&maps.k, a.pg.k_code, kMapBytes, D, rows, D, box, D, 256) ||
      !make_tensor_map_2d(&maps.v, a.pg.v_code, kMapBytes, D, rows, D, box, D, 256))
    return cudaErrorInvalidValue;
  const size_t smem = (size_t)kWarps * kRingBytes + 1024;
  auto kern = paged_attend_kernel<T, D, RL, F32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kern, dim3(p.n_warps / kWarps), kWarps * 32, smem, s, p, maps);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_combine_kernel<T, D>, dim3(a.n_q * a.Hq, a.pg.n_seqs),
                          kCombineThreads, 0, s, p);
}

template <typename T, int D, bool F32>
cudaError_t attend_d(const AttendParams& p, cudaStream_t s) {
  if (p.rp.rows == 4) return attend_t<T, D, 1, F32>(p, s);
  if constexpr (!F32)
    if (p.rp.rows == 16) return attend_t<T, D, 4, F32>(p, s);
  return attend_t<T, D, 2, F32>(p, s);
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
  p.n_warps = (num_sms < kMaxCtas ? num_sms : kMaxCtas) * kWarps;
  p.ws = ws_layout(a.ws, a.H, p.rp, a.d, a.pg.n_seqs, nullptr);
  if (a.dtype == LOWRAM_DTYPE_BF16)
    return a.d == 128 ? attend_d<__nv_bfloat16, 128, false>(p, s)
                      : attend_d<__nv_bfloat16, 64, false>(p, s);
  return a.d == 128 ? attend_d<float, 128, true>(p, s)
                    : attend_d<float, 64, true>(p, s);
}

}  // namespace lowram
