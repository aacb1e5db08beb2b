// norm.cu -- root-mean-square norm with the residual's addition and FP8
// output, and its backward pass.  sm_100a only.
//
// Forward, per row:
//   h = x + residual,  rstd = 1 / sqrt(mean(h^2) + eps),  y = (h w) rstd,
//   m = fmax / max|y| per row or per block of columns,  q = RNE(y m)
// One reduction serves both statistics: rstd > 0 is one factor for the row
// and rounding is monotone, so max|y| = max|h w| * rstd exactly, and the sum
// of squares and the maxima of |h w| are taken together.
//
// Backward, per row, with xh = h rstd and gw = dy w:
//   dx = dres + rstd (gw - xh mean(gw xh)),   dw += dy xh
// Each CTA adds dw over its rows (in row order) and writes one partial row
// of f32 sums; a second launch adds the CTAs' partials in CTA order, so the
// sum has a fixed order and the workspace needs no initial state.
//
// Bound: memory where a row brings two tensors or more ([16384, 8192] bf16
// with a residual: 144 us replayed from a graph, 161 in calls among others, 6.5
// and 5.8 TB/s; backward 156 and 165 us, 6.9 and 6.5 TB/s, part of it from
// L2), the latency of the row's serial steps (sum, maximum, divisions) with
// few rows in flight for one tensor a row (93 us, 4.3 TB/s).
#include "elem.cuh"
#include "fp8_cvt.cuh"
#include "hq_internal.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "row_grid.cuh"

#include <atomic>

namespace hq {
namespace {

constexpr uint32_t kInfBits = 0x7F800000u;
constexpr int kNormMaxBlocks = static_cast<int>(kNormMaxCols / 16);

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// fmax / amax, 1 when amax is 0 or the quotient is not finite
__device__ __forceinline__ float multiplier_of(float amax, int fmt) {
  if (!(amax > 0.0f)) return 1.0f;
  const float m = __fdiv_rn(fmt == 0 ? kFmaxE4M3 : kFmaxE5M2, amax);
  return (m <= FLT_MAX) ? m : 1.0f;
}

__device__ __forceinline__ uint8_t encode_rt(float y, int fmt) { return fmt == 0 ? cvt1_exact<0>(y) : cvt1_exact<1>(y); }

// Sum of v and maximum of mx over the CTA; red: 2 x 33 words.
template <int THREADS>
__device__ __forceinline__ void cta_sum_max(float& v, uint32_t& mx, float* red) {
  v = warp_sum(v);
  mx = __reduce_max_sync(0xFFFFFFFFu, mx);
  uint32_t* redm = reinterpret_cast<uint32_t*>(red + 33);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5] = v;
    redm[threadIdx.x >> 5] = mx;
  }
  __syncthreads();
  v = 0.0f;
  mx = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    v += red[w];
    mx = max(mx, redm[w]);
  }
}

struct NormParams {
  const void* x;
  const void* residual;
  const void* weight;
  int wt;
  int rows, cols;
  float eps;
  int fmt;
  int block, nb;     // block 0: one scale per row
  uint8_t* q;
  float* scales;
  void* residual_out;
  void* y_out;
  float* rstd_out;
};

// ------------------------------------------------------------ any layout
// One CTA per row at a time, one element per access, the row read twice (a
// third time when it holds an infinity or NaN): what the kernels on vectors
// do not take -- buffers that start off 16-byte boundaries, rows of less than
// three vectors between them, blocks that are no power of two of vectors up
// to 32.
constexpr int kAnyThreads = 256;

template <int XT>
__global__ void __launch_bounds__(kAnyThreads) k_rmsnorm_any(const NormParams p) {
  __shared__ float red[66];
  __shared__ uint32_t bmax[kNormMaxBlocks];  // per block: bits of max|h w|, then the multiplier
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t base = row * p.cols;
    auto load_h = [&](int c) {
      float h = elem_load<XT>(p.x, base + c);
      if (p.residual) h = __fadd_rn(h, elem_load<XT>(p.residual, base + c));
      return h;
    };
    auto clear_blocks = [&] {
      for (int b = tid; b < p.nb; b += kAnyThreads) bmax[b] = 0u;
      __syncthreads();
    };
    __syncthreads();  // the previous row's multipliers are read out
    clear_blocks();
    float ss = 0.0f;
    uint32_t mx = 0;
    for (int c = tid; c < p.cols; c += kAnyThreads) {
      const float h = load_h(c);
      ss = fmaf(h, h, ss);
      const uint32_t a = __float_as_uint(__fmul_rn(h, elem_load_rt(p.weight, p.wt, c))) & 0x7FFFFFFFu;
      mx = max(mx, a);
      if (p.block) atomicMax(&bmax[c / p.block], a);
    }
    cta_sum_max<kAnyThreads>(ss, mx, red);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(p.cols)), p.eps)));
    float top = __fmul_rn(__uint_as_float(mx), rstd);  // max|y|; not finite: some y may be
    const bool special = mx >= kInfBits || !(top <= FLT_MAX);
    if (special) {  // amax over the finite |y| alone
      clear_blocks();
      float am = 0.0f;
      for (int c = tid; c < p.cols; c += kAnyThreads) {
        const float y = finite_abs(__fmul_rn(__fmul_rn(load_h(c), elem_load_rt(p.weight, p.wt, c)), rstd));
        am = fmaxf(am, y);
        if (p.block) atomicMax(&bmax[c / p.block], __float_as_uint(y));
      }
      float zero = 0.0f;
      uint32_t ab = __float_as_uint(am);
      cta_sum_max<kAnyThreads>(zero, ab, red);
      top = __uint_as_float(ab);
    }
    float m = 1.0f;
    if (p.block) {
      for (int b = tid; b < p.nb; b += kAnyThreads) {
        const float a = __uint_as_float(bmax[b]);
        const float mb = multiplier_of(special ? a : __fmul_rn(a, rstd), p.fmt);
        p.scales[row * p.nb + b] = __fdiv_rn(1.0f, mb);
        bmax[b] = __float_as_uint(mb);
      }
      __syncthreads();
    } else {
      m = multiplier_of(top, p.fmt);
      if (tid == 0) p.scales[row] = __fdiv_rn(1.0f, m);
    }
    if (tid == 0 && p.rstd_out) p.rstd_out[row] = rstd;
    for (int c = tid; c < p.cols; c += kAnyThreads) {
      const float h = load_h(c);
      const float y = __fmul_rn(__fmul_rn(h, elem_load_rt(p.weight, p.wt, c)), rstd);
      if (p.residual_out) elem_store<XT>(p.residual_out, base + c, h);
      if (p.y_out) elem_store<XT>(p.y_out, base + c, y);
      p.q[base + c] = encode_rt(__fmul_rn(y, p.block ? __uint_as_float(bmax[c / p.block]) : m), p.fmt);
    }
  }
}

// ------------------------------------------------------- 16-byte vectors
// A CTA takes rows blockIdx.x, + gridDim.x, ...; bulk copies (TMA) bring the
// next rows of x and residual into a ring of shared-memory stages, thread t
// holds E elements of the row (16-byte vectors t, t + T, ..) and its share
// of the weight in registers.  One block barrier per row joins the sum of
// squares and the maximum; behind it every thread has read the row's stage,
// so the refill needs no barrier of its own.
//
// Block-wise scales: a block of 16-byte vectors that is a power of two up to
// 32 lies inside one warp's consecutive lanes, so its maximum is a shuffle, and
// its lanes share out the divisions of the blocks that they hold.
constexpr int kRingStages = 8;
// Elements per thread.  Most rows run with 16 or 24 elements and the weight
// in registers, up to 512 threads of 128 registers per SM: measured on
// [16384, 8192] bf16 with a residual, 16 elements in one CTA of 512 threads
// took 148 us, held to 64 registers with two CTAs 171 us (the compiler then
// orders the loads behind one another), 32 elements in two CTAs of 256
// threads 171 us, in one 190 us; the backward pass 158, 180, 165 and 164 us.
// Eight elements serve a single row per CTA (latency) and narrow rows.
//
// Rows beyond the columns or the stages of one CTA are split over a cluster
// (CL): every CTA a run of the row's vectors, the warps' sums and maxima
// written into all its CTAs' shared memories, a cluster barrier in place of
// the block's: [4096, 28672] f32 292 us forward and 427 backward, against 977
// and 2305 with one element per access.
constexpr int kRingMaxCols = 16384;
constexpr int ring_max_threads(int e) { return e == 8 ? 1024 : 512; }
constexpr int kRingSlots = 64;  // warps of a CTA or cluster

template <int XT>
constexpr int vec_elems() {
  return XT == 0 ? 4 : 8;
}
// vectors that a row of cols columns touches, at most, wherever it starts
template <int VEC>
__host__ __device__ constexpr uint32_t shifted_vecs(int cols) {
  return static_cast<uint32_t>((cols + 2 * VEC - 2) / VEC);
}
// vectors of a row per CTA of its cluster: whole blocks of scales in each
template <int VEC, bool SHIFT>
__host__ __device__ constexpr int cluster_share(int cols, int ctas) {
  const int all = SHIFT ? static_cast<int>(shifted_vecs<VEC>(cols)) : cols / VEC;
  return ((all + ctas - 1) / ctas + 31) / 32 * 32;
}

struct RingShared {
  uint64_t full[kRingStages];
  float sum[2][kRingSlots];       // by row parity, per warp of the CTA (or cluster)
  uint32_t top[2][kRingSlots];
  int abort_flag;
};

constexpr uint32_t kGaveUp = 0xFFFFFFFFu;  // above every maximum's bits

__device__ __forceinline__ void ring_init(RingShared& sh, int stages) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) ptx::mbar_init(&sh.full[s], 1);
    sh.abort_flag = 0;
    ptx::fence_mbarrier_init();
  }
  __syncthreads();
}

// After a wait that gave up at `stage` (of parity `phase`): the copies still
// in flight into this CTA's shared memory land, or the drain limit passes,
// before it leaves.  Stages from `stage` on, up to and without next_stage,
// hold rows not yet waited for; where the two are equal, all of them may.
// A stage that was not filled again has nothing in flight: its
// wait ends at the limit.
__device__ __forceinline__ void drain_stages(uint64_t* full, int stages, int stage, uint32_t phase, int next_stage) {
  int dummy = 0;
  do {
    ptx::mbar_wait(&full[stage], phase, &dummy, nullptr, 0, ptx::kDrainLimitNs);
    if (++stage == stages) { stage = 0; phase ^= 1u; }
  } while (stage != next_stage);
}

// the warps' values joined (after the barrier); CL: up to 64 of them
template <bool CL>
__device__ __forceinline__ float join_sum(const float* red, int warps) {
  const int lane = threadIdx.x & 31;
  float v = lane < warps ? red[lane] : 0.0f;
  if (CL && lane + 32 < warps) v += red[lane + 32];
  return warp_sum(v);
}
template <bool CL>
__device__ __forceinline__ uint32_t join_max(const uint32_t* red, int warps) {
  const int lane = threadIdx.x & 31;
  uint32_t v = lane < warps ? red[lane] : 0u;
  if (CL && lane + 32 < warps) v = max(v, red[lane + 32]);
  return __reduce_max_sync(0xFFFFFFFFu, v);
}

// Rows that start between 16-byte boundaries (SHIFT, a width that is not a
// whole number of vectors): the row's vectors are those of the whole tensor,
// the first and last of them shared with the neighbouring rows.  A CTA's (or
// team's) rows lie a multiple of VEC rows apart, so that they all start at
// the same place of a vector and the columns that a thread holds, its weights
// and its sums of dw stay the same: [16384, 1001] bf16 31.2 us forward and
// 34.0 backward, against 180 and 372 with one element per access.
// Where the tensor ends inside a row's last vector, the CTA's first thread
// copies the elements before that end into the stage itself.
// These helpers keep to few registers: they sit in the kernels' inner loops.
template <int VEC>
__device__ __forceinline__ bool is_edge(int c0, int cols) {
  return c0 < 0 || c0 + VEC > cols;
}
// zero in the columns of other rows; the vector starts at column c0
template <int XT>
__device__ __forceinline__ void mask_edge(uint4& u, int c0, int cols) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (XT == 0) {
      if (static_cast<unsigned>(c0 + k) >= static_cast<unsigned>(cols)) w[k] = 0;
    } else {
      if (static_cast<unsigned>(c0 + 2 * k) >= static_cast<unsigned>(cols)) w[k] &= 0xFFFF0000u;
      if (static_cast<unsigned>(c0 + 2 * k + 1) >= static_cast<unsigned>(cols)) w[k] &= 0x0000FFFFu;
    }
  }
}
// the elements of N packed ones of BYTES that are this row's; at: address of column c0
template <int BYTES, int N>
__device__ __forceinline__ void store_edge(void* at, int c0, int cols, const uint32_t* w) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t e = w[j * BYTES / 4] >> (8 * (j * BYTES % 4));
    if (static_cast<unsigned>(c0 + j) < static_cast<unsigned>(cols)) {
      if (BYTES == 1) static_cast<uint8_t*>(at)[j] = static_cast<uint8_t>(e);
      else if (BYTES == 2) static_cast<uint16_t*>(at)[j] = static_cast<uint16_t>(e);
      else static_cast<uint32_t*>(at)[j] = e;
    }
  }
}
template <int XT>
__device__ __forceinline__ void store_edge_vec(void* at, int c0, int cols, const uint4& u) {
  store_edge<elem_bytes<XT>(), vec_elems<XT>()>(at, c0, cols, reinterpret_cast<const uint32_t*>(&u));
}
// the n elements before the tensor's end, into the last vector of a stage's row
template <int XT>
__device__ __forceinline__ void copy_tail(void* to, const void* from, int n) {
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    if (XT == 0) static_cast<float*>(to)[j] = static_cast<const volatile float*>(from)[j];
    else static_cast<uint16_t*>(to)[j] = static_cast<const volatile uint16_t*>(from)[j];
  }
}
// A thread's weights (element type code WT) as f32: vectors tid, tid + T, ...
// of the nv from column col0.  SHIFT: element by element, zero in other rows'
// columns.  All loads are in flight together, so nothing about them branches:
// indices past the row are held at its last (with a branch per element the
// loads came one after the other, 8 us of a [37, 12307] call's 11).
template <int WT, int VEC, int ITEMS, bool SHIFT>
__device__ __forceinline__ void load_weights_as(const void* w, int col0, int cols, int nv, int tid, int T, float* f) {
#pragma unroll
  for (int it = 0; it < ITEMS; ++it) {
    const int c0 = col0 + min(it * T + tid, nv - 1) * VEC;
    float* o = f + it * VEC;
    if (SHIFT) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int c = c0 + j;
        const float e = elem_load_rt(w, WT, max(0, min(c, cols - 1)));
        o[j] = c >= 0 && c < cols ? e : 0.0f;
      }
    } else if (WT == 0) {
#pragma unroll
      for (int j = 0; j < VEC; j += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + c0 + j));
        o[j] = v.x; o[j + 1] = v.y; o[j + 2] = v.z; o[j + 3] = v.w;
      }
    } else {
      uint4 u = make_uint4(0, 0, 0, 0);
      const unsigned short* ws = static_cast<const unsigned short*>(w) + c0;
      if (VEC == 8) {
        u = __ldg(reinterpret_cast<const uint4*>(ws));
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(ws));
        u.x = v.x; u.y = v.y;
      }
      float t[8];
      vec_widen<WT>(u, t);
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = t[j];
    }
  }
}
template <int VEC, int ITEMS, bool SHIFT>
__device__ __forceinline__ void load_weights(const void* w, int wt, int col0, int cols, int nv, int tid, int T, float2* f) {
  float* o = reinterpret_cast<float*>(f);
  if (wt == 0) load_weights_as<0, VEC, ITEMS, SHIFT>(w, col0, cols, nv, tid, T, o);
  else if (wt == 1) load_weights_as<1, VEC, ITEMS, SHIFT>(w, col0, cols, nv, tid, T, o);
  else load_weights_as<2, VEC, ITEMS, SHIFT>(w, col0, cols, nv, tid, T, o);
}

// VEC codes of y * m; EXACT: y may hold NaN
template <int VEC, int FMT, bool EXACT>
__device__ __forceinline__ void codes_as(uint32_t (&c)[VEC / 4], const float2* y, float m) {
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    const float2 t = f2_mul(y[j], make_float2(m, m));
    const uint32_t c2 = EXACT ? cvt2_exact<FMT>(t.x, t.y) : cvt2_fast<FMT>(t.x, t.y);
    c[j / 2] = (j & 1) ? (c[j / 2] | (c2 << 16)) : c2;
  }
}
template <int VEC>
__device__ __forceinline__ void codes(uint32_t (&c)[VEC / 4], const float2* y, float m, int fmt, bool exact) {
  if (exact) {
    if (fmt == 0) codes_as<VEC, 0, true>(c, y, m);
    else codes_as<VEC, 1, true>(c, y, m);
  } else {
    if (fmt == 0) codes_as<VEC, 0, false>(c, y, m);
    else codes_as<VEC, 1, false>(c, y, m);
  }
}

template <int XT, int E, bool RES, bool SHIFT, bool CL>
__global__ void __launch_bounds__(ring_max_threads(E), 1) k_rmsnorm_ring(const NormParams p, const int stages, unsigned* err) {
  constexpr int VEC = vec_elems<XT>();
  constexpr int ITEMS = E / VEC;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ RingShared sh;
  const int tid = threadIdx.x, T = blockDim.x;
  const int warp = tid >> 5, lane = tid & 31, warps = T >> 5;
  const int ctas = CL ? static_cast<int>(ptx::cluster_size()) : 1, rank = CL ? static_cast<int>(ptx::cluster_rank()) : 0;
  const int first = CL ? static_cast<int>(blockIdx.x) / ctas : static_cast<int>(blockIdx.x);
  const int stride = CL ? static_cast<int>(gridDim.x) / ctas : static_cast<int>(gridDim.x);
  // columns before the row in its first vector; the same for all rows of a CTA
  const int shift = SHIFT ? static_cast<int>(static_cast<int64_t>(first) * p.cols % VEC) : 0;
  const int all = (shift + p.cols + VEC - 1) / VEC;
  const int share = CL ? cluster_share<VEC, SHIFT>(p.cols, ctas) : all;  // vectors per CTA
  const int nv = CL ? max(0, min(share, all - rank * share)) : all;
  const int col0 = (CL ? rank * share * VEC : 0) - shift;  // this CTA's first column
  const int slots = (T >> 5) * ctas;
  // room in a stage
  const uint32_t row_bytes = CL ? share * 16u : SHIFT ? shifted_vecs<VEC>(p.cols) * 16u : static_cast<uint32_t>(nv) * 16u;
  const uint32_t stage_bytes = row_bytes * (RES ? 2 : 1);
  const int64_t total = static_cast<int64_t>(p.rows) * p.cols;
  ring_init(sh, stages);
  if (CL) ptx::cluster_barrier();  // all CTAs of the cluster are there to be written to
  pdl_wait();
  pdl_launch_dependents();
  int next = first;  // thread 0: the next row to bring in, and its stage
  int next_stage = 0;
  auto issue = [&] {
    const int s = next_stage;
    const int64_t at = static_cast<int64_t>(next) * p.cols + col0;  // a multiple of VEC
    const char* x = static_cast<const char*>(p.x) + at * elem_bytes<XT>();
    const char* r = RES ? static_cast<const char*>(p.residual) + at * elem_bytes<XT>() : nullptr;
    uint8_t* to = ring + s * stage_bytes;
    uint32_t bytes = nv * 16u;
    if (SHIFT && at + static_cast<int64_t>(nv) * VEC > total) {
      bytes -= 16;
      const int n = static_cast<int>(total - at) - (nv - 1) * VEC;
      copy_tail<XT>(to + bytes, x + bytes, n);
      if (RES) copy_tail<XT>(to + row_bytes + bytes, r + bytes, n);
    }
    ptx::mbar_arrive_expect_tx(&sh.full[s], bytes * (RES ? 2 : 1));
    ptx::bulk_load(to, x, bytes, &sh.full[s]);
    if (RES) ptx::bulk_load(to + row_bytes, r, bytes, &sh.full[s]);
    next = p.rows - next > stride ? next + stride : p.rows;  // no overflow near 2^31 rows
    if (++next_stage == stages) next_stage = 0;
  };
  if (tid == 0)
    for (int s = 0; s < stages && next < p.rows; ++s) issue();
  const float inv_cols = __fdiv_rn(1.0f, static_cast<float>(p.cols));
  float2 w[E / 2];
  load_weights<VEC, ITEMS, SHIFT>(p.weight, p.wt, col0, p.cols, nv, tid, T, w);
  const int group = p.block ? p.block / VEC : 0;  // lanes per block, a power of two
  const int group_log = 31 - __clz(group | 1);
  int stage = 0;
  uint32_t phase = 0;
  int par = 0;
  bool quit = false;
  for (int row = first; row < p.rows; row = p.rows - row > stride ? row + stride : p.rows) {
    const bool ok = ptx::mbar_wait_inline(&sh.full[stage], phase, &sh.abort_flag, err, kDevErrTimeout);
    const uint4* xs = reinterpret_cast<const uint4*>(ring + stage * stage_bytes);
    const uint4* rs = reinterpret_cast<const uint4*>(ring + stage * stage_bytes + row_bytes);
    const int64_t row_at = static_cast<int64_t>(row) * p.cols;
    // every vector is asked for before the first is used
    uint4 xr[ITEMS], rr[RES ? ITEMS : 1];
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const int v = it * T + tid;
      if (v < nv) {
        xr[it] = xs[v];
        if (RES) rr[RES ? it : 0] = rs[v];
      }
    }
    float2 h[E / 2];
    float2 ss2 = make_float2(0.0f, 0.0f);
    float vtop[ITEMS], top = 0.0f;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const int v = it * T + tid;
      float2* hv = h + it * (VEC / 2);
      vtop[it] = 0.0f;
      if (v < nv) {
        const int c0 = col0 + v * VEC;
        const bool edge = SHIFT && is_edge<VEC>(c0, p.cols);
        if (SHIFT && edge) {
          mask_edge<XT>(xr[it], c0, p.cols);
          if (RES) mask_edge<XT>(rr[RES ? it : 0], c0, p.cols);
        }
        vec_widen<XT>(xr[it], reinterpret_cast<float*>(hv));
        if (RES) {
          float2 r[VEC / 2];
          vec_widen<XT>(rr[RES ? it : 0], reinterpret_cast<float*>(r));
#pragma unroll
          for (int j = 0; j < VEC / 2; ++j) hv[j] = f2_add(hv[j], r[j]);
          if (p.residual_out) {
            const uint4 u = vec_narrow<XT>(reinterpret_cast<const float*>(hv));
            char* to = static_cast<char*>(p.residual_out) + (row_at + c0) * elem_bytes<XT>();
            if (SHIFT && edge) store_edge_vec<XT>(to, c0, p.cols, u);
            else vec_store(to, u);
          }
        }
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          ss2 = f2_fma(hv[j], hv[j], ss2);
          hv[j] = f2_mul(hv[j], w[it * (VEC / 2) + j]);  // h w from here on
          vtop[it] = max3_abs_nan(vtop[it], hv[j].x, hv[j].y);
        }
        top = max3_abs_nan(top, vtop[it], 0.0f);
      } else {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) hv[j] = make_float2(0.0f, 0.0f);
      }
    }
    float ss = warp_sum(ss2.x + ss2.y);
    const uint32_t wtop = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));  // NaN's bits are above infinity's
    if (CL) {
      const bool gave_up = __any_sync(0xFFFFFFFFu, !ok);
      if (lane < ctas) {
        const int slot = rank * warps + warp;
        ptx::store_cluster(&sh.sum[par][slot], lane, __float_as_uint(ss));
        ptx::store_cluster(&sh.top[par][slot], lane, gave_up ? kGaveUp : wtop);
      }
      ptx::cluster_barrier();
    } else {
      if (lane == 0) {
        sh.sum[par][warp] = ss;
        sh.top[par][warp] = wtop;
      }
      quit = __syncthreads_or(!ok) != 0;  // the whole CTA agrees on giving up
      if (quit) break;
      if (tid == 0 && next < p.rows) issue();
    }
    ss = join_sum<CL>(sh.sum[par], slots);
    const uint32_t tbits = join_max<CL>(sh.top[par], slots);
    if (CL) {
      quit = tbits == kGaveUp;  // so does the cluster
      if (quit) break;
      if (tid == 0 && next < p.rows) issue();
    }
    const float rstd = rsqrtf(fmaf(ss, inv_cols, p.eps));
    float amax = __fmul_rn(__uint_as_float(tbits), rstd);
    const bool special = tbits >= kInfBits || !(amax <= FLT_MAX);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) h[e] = f2_mul(h[e], make_float2(rstd, rstd));  // y
    if (special) {  // amax over the finite |y| alone
      float fin = 0.0f;
#pragma unroll
      for (int it = 0; it < ITEMS; ++it) {
        float vt = 0.0f;
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j)
          vt = fmaxf(vt, fmaxf(finite_abs(h[it * (VEC / 2) + j].x), finite_abs(h[it * (VEC / 2) + j].y)));
        vtop[it] = vt;
        fin = fmaxf(fin, vt);
      }
      const uint32_t wfin = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fin));
      // everyone has read this row's maxima, then they are the finite ones
      if (CL) {
        ptx::cluster_barrier();
        if (lane < ctas) ptx::store_cluster(&sh.top[par][rank * warps + warp], lane, wfin);
        ptx::cluster_barrier();
      } else {
        __syncthreads();
        if (lane == 0) sh.top[par][warp] = wfin;
        __syncthreads();
      }
      amax = __uint_as_float(join_max<CL>(sh.top[par], slots));
    }
    if (tid == 0 && rank == 0 && p.rstd_out) p.rstd_out[row] = rstd;
    float m[ITEMS];
    if (group == 0) {
      m[0] = multiplier_of(amax, p.fmt);
      if (tid == 0 && rank == 0) p.scales[row] = __fdiv_rn(1.0f, m[0]);
#pragma unroll
      for (int it = 1; it < ITEMS; ++it) m[it] = m[0];
    } else {
      for (int o = 1; o < group; o <<= 1) {
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) vtop[it] = fmaxf(vtop[it], __shfl_xor_sync(0xFFFFFFFFu, vtop[it], o));
      }
      float* srow = p.scales + static_cast<int64_t>(row) * p.nb + (CL ? rank * (share >> group_log) : 0);
      const int in = lane & (group - 1);
      if (group >= ITEMS) {  // lane `in` of a group divides for the group's block of item `in`
        float mine = vtop[0];
#pragma unroll
        for (int it = 1; it < ITEMS; ++it) mine = in == it ? vtop[it] : mine;
        const float mb = multiplier_of(special ? mine : __fmul_rn(mine, rstd), p.fmt);
        const float inv = __fdiv_rn(1.0f, mb);
        const int v = in * T + tid;
        if (in < ITEMS && v - in < nv) srow[v >> group_log] = inv;
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) m[it] = __shfl_sync(0xFFFFFFFFu, mb, lane - in + it);
      } else {
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
          const int v = it * T + tid;
          m[it] = multiplier_of(special ? vtop[it] : __fmul_rn(vtop[it], rstd), p.fmt);
          if (in == 0 && v < nv) srow[v >> group_log] = __fdiv_rn(1.0f, m[it]);
        }
      }
    }
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const int v = it * T + tid;
      if (v < nv) {
        const int c0 = col0 + v * VEC;
        const int64_t at = row_at + c0;
        const float2* y = h + it * (VEC / 2);
        uint32_t c4[VEC / 4];
        codes<VEC>(c4, y, m[it], p.fmt, special);
        char* yo = static_cast<char*>(p.y_out) + at * elem_bytes<XT>();
        if (SHIFT && is_edge<VEC>(c0, p.cols)) {
          if (p.y_out) store_edge_vec<XT>(yo, c0, p.cols, vec_narrow<XT>(reinterpret_cast<const float*>(y)));
          store_edge<1, VEC>(p.q + at, c0, p.cols, c4);
        } else {
          if (p.y_out) vec_store(yo, vec_narrow<XT>(reinterpret_cast<const float*>(y)));
          if (VEC == 8) *reinterpret_cast<uint2*>(p.q + at) = make_uint2(c4[0], c4[VEC / 4 - 1]);
          else *reinterpret_cast<uint32_t*>(p.q + at) = c4[0];
        }
      }
    }
    if (++stage == stages) { stage = 0; phase ^= 1u; }
    par ^= 1;
  }
  if (quit) {
    if (tid == 0) drain_stages(sh.full, stages, stage, phase, next_stage);
    __syncthreads();
  }
}

struct NormBwdParams {
  const void* dy;
  const void* h;
  const void* dres;
  const void* weight;
  int wt;
  const float* rstd;
  int rows, cols;
  void* dx;
  float* part;   // [gridDim.x, cols] or null
};

constexpr int kBwdParts = 296;  // two CTAs per SM
constexpr int kTeams = 15;      // teams of a backward CTA at most (barriers 1 .. 15)

// CTA b takes rows b, b + grid, ...; dw sums in shared memory, one slot per
// column, each touched by one thread only.
template <int XT>
__global__ void __launch_bounds__(kAnyThreads) k_rmsnorm_bwd_any(const NormBwdParams p) {
  extern __shared__ float dw[];
  __shared__ float red[66];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  if (p.part)
    for (int c = tid; c < p.cols; c += kAnyThreads) dw[c] = 0.0f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t base = row * p.cols;
    const float rs = __ldg(p.rstd + row);
    float dot = 0.0f;
    for (int c = tid; c < p.cols; c += kAnyThreads)
      dot = fmaf(elem_load<XT>(p.dy, base + c) * elem_load_rt(p.weight, p.wt, c), elem_load<XT>(p.h, base + c) * rs, dot);
    uint32_t none = 0;
    cta_sum_max<kAnyThreads>(dot, none, red);
    const float mean = __fdiv_rn(dot, static_cast<float>(p.cols));
    for (int c = tid; c < p.cols; c += kAnyThreads) {
      const float g = elem_load<XT>(p.dy, base + c);
      const float xh = elem_load<XT>(p.h, base + c) * rs;
      float d = rs * fmaf(-xh, mean, g * elem_load_rt(p.weight, p.wt, c));
      if (p.dres) d += elem_load<XT>(p.dres, base + c);
      elem_store<XT>(p.dx, base + c, d);
      if (p.part) dw[c] = fmaf(g, xh, dw[c]);
    }
  }
  if (p.part)
    for (int c = tid; c < p.cols; c += kAnyThreads) p.part[static_cast<int64_t>(blockIdx.x) * p.cols + c] = dw[c];
}

// Barrier of one team of T threads (a power of two of them share a CTA), and
// whether any of its threads says so.
__device__ __forceinline__ bool team_any(int team, int T, bool say) {
  if (T == 32) return __any_sync(0xFFFFFFFFu, say);
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
      "barrier.cta.red.or.pred.aligned p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(team + 1), "r"(T), "r"(say ? 1u : 0u)
      : "memory");
  return r != 0;
}

// 16-byte rows: the forward kernel's ring over dy, h and dres.  A CTA is
// `teams` teams of T threads with a row and a ring each (narrow rows: enough
// rows in flight without a partial row of dw per row).  Both passes over a
// row (the mean, then dx and dw) read its stage, so the stage of row i is
// refilled after row i + 1's barrier (two stages at least, or one row).  dw stays in registers; the teams'
// sums join in order through shared memory.
template <int XT, int E, bool DRES, bool SHIFT, bool CL>
__global__ void __launch_bounds__(ring_max_threads(E), 1)
    k_rmsnorm_bwd_ring(const NormBwdParams p, const int teams, const int stages, unsigned* err) {
  constexpr int VEC = vec_elems<XT>();
  constexpr int ITEMS = E / VEC;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kTeams][kRingStages];
  __shared__ float sums[2][kRingSlots];  // by row parity, per warp of the CTA (or cluster)
  __shared__ uint32_t gave_up[2][kRingSlots];  // CL: which of them gave up a wait
  __shared__ int abort_flag;
  const int T = blockDim.x / teams;
  const int team = threadIdx.x / T, tid = threadIdx.x - team * T;
  const int lane = tid & 31, warps = T >> 5;
  // rows of this team: first, first + stride, .. (grid and teams are small: all in int)
  const int ctas = CL ? static_cast<int>(ptx::cluster_size()) : 1, rank = CL ? static_cast<int>(ptx::cluster_rank()) : 0;
  const int unit = CL ? static_cast<int>(blockIdx.x) / ctas : static_cast<int>(blockIdx.x);
  const int first = unit * teams + team;
  const int stride = (CL ? static_cast<int>(gridDim.x) / ctas : static_cast<int>(gridDim.x)) * teams;
  // columns before the row in its first vector; the same for all rows of a team
  const int shift = SHIFT ? static_cast<int>(static_cast<int64_t>(first) * p.cols % VEC) : 0;
  const int all = (shift + p.cols + VEC - 1) / VEC;
  const int share = CL ? cluster_share<VEC, SHIFT>(p.cols, ctas) : all;  // vectors per CTA
  const int nv = CL ? max(0, min(share, all - rank * share)) : all;
  const int col0 = (CL ? rank * share * VEC : 0) - shift;  // this CTA's first column
  // room in a stage
  const uint32_t row_bytes = CL ? share * 16u : SHIFT ? shifted_vecs<VEC>(p.cols) * 16u : static_cast<uint32_t>(nv) * 16u;
  const uint32_t stage_bytes = row_bytes * (DRES ? 3 : 2);
  const int64_t total = static_cast<int64_t>(p.rows) * p.cols;
  uint8_t* ring = smem + team * stages * stage_bytes;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) ptx::mbar_init(&full[team][s], 1);
    if (team == 0) abort_flag = 0;
    ptx::fence_mbarrier_init();
  }
  __syncthreads();
  if (CL) ptx::cluster_barrier();  // all CTAs of the cluster are there to be written to
  pdl_wait();
  pdl_launch_dependents();
  int next = first;  // thread 0: the next row to bring in, and its stage
  int next_stage = 0;
  auto issue = [&] {
    const int s = next_stage;
    const int64_t at = static_cast<int64_t>(next) * p.cols + col0;  // a multiple of VEC
    const int64_t off = at * elem_bytes<XT>();
    uint8_t* to = ring + s * stage_bytes;
    uint64_t* bar = &full[team][s];
    uint32_t bytes = nv * 16u;
    if (SHIFT && at + static_cast<int64_t>(nv) * VEC > total) {
      bytes -= 16;
      const int n = static_cast<int>(total - at) - (nv - 1) * VEC;
      copy_tail<XT>(to + bytes, static_cast<const char*>(p.dy) + off + bytes, n);
      copy_tail<XT>(to + row_bytes + bytes, static_cast<const char*>(p.h) + off + bytes, n);
      if (DRES) copy_tail<XT>(to + 2 * row_bytes + bytes, static_cast<const char*>(p.dres) + off + bytes, n);
    }
    ptx::mbar_arrive_expect_tx(bar, bytes * (DRES ? 3 : 2));
    ptx::bulk_load(to, static_cast<const char*>(p.dy) + off, bytes, bar);
    ptx::bulk_load(to + row_bytes, static_cast<const char*>(p.h) + off, bytes, bar);
    if (DRES) ptx::bulk_load(to + 2 * row_bytes, static_cast<const char*>(p.dres) + off, bytes, bar);
    next = p.rows - next > stride ? next + stride : p.rows;  // no overflow near 2^31 rows
    if (++next_stage == stages) next_stage = 0;
  };
  if (tid == 0)
    for (int s = 0; s < stages && next < p.rows; ++s) issue();
  const float inv_cols = __fdiv_rn(1.0f, static_cast<float>(p.cols));
  float2 w[E / 2], dw[E / 2];
  load_weights<VEC, ITEMS, SHIFT>(p.weight, p.wt, col0, p.cols, nv, tid, T, w);
#pragma unroll
  for (int j = 0; j < E / 2; ++j) dw[j] = make_float2(0.0f, 0.0f);
  float rs_next = first < p.rows ? __ldg(p.rstd + first) : 0.0f;
  int stage = 0;
  uint32_t phase = 0;
  bool ahead = false;  // a row of this team is done
  bool quit = false;
  int par = 0;
  for (int row = first; row < p.rows;) {
    const float rs = rs_next;
    const int row_next = p.rows - row > stride ? row + stride : p.rows;
    if (row_next < p.rows) rs_next = __ldg(p.rstd + row_next);
    const bool ok = ptx::mbar_wait_inline(&full[team][stage], phase, &abort_flag, err, kDevErrTimeout);
    const uint4* gs = reinterpret_cast<const uint4*>(ring + stage * stage_bytes);
    const uint4* hs = reinterpret_cast<const uint4*>(ring + stage * stage_bytes + row_bytes);
    const uint4* ds = reinterpret_cast<const uint4*>(ring + stage * stage_bytes + 2 * row_bytes);
    const int64_t row_at = static_cast<int64_t>(row) * p.cols;
    auto fetch = [&](const uint4* stage_row, int v, float2* f) {
      uint4 u = stage_row[v];
      if (SHIFT && is_edge<VEC>(col0 + v * VEC, p.cols)) mask_edge<XT>(u, col0 + v * VEC, p.cols);
      vec_widen<XT>(u, reinterpret_cast<float*>(f));
    };
    const float2 rs2 = make_float2(rs, rs);
    float2 dot2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const int v = it * T + tid;
      if (v < nv) {
        float2 g[VEC / 2], h[VEC / 2];
        fetch(gs, v, g);
        fetch(hs, v, h);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) dot2 = f2_fma(f2_mul(g[j], w[it * (VEC / 2) + j]), h[j], dot2);
      }
    }
    float dot = warp_sum(dot2.x + dot2.y);
    if (CL) {
      const bool out_of_time = __any_sync(0xFFFFFFFFu, !ok);
      if (lane < ctas) {
        const int slot = rank * warps + static_cast<int>(threadIdx.x >> 5);
        ptx::store_cluster(&sums[par][slot], lane, __float_as_uint(dot));
        ptx::store_cluster(&gave_up[par][slot], lane, out_of_time ? kGaveUp : 0u);
      }
      ptx::cluster_barrier();
      quit = join_max<true>(gave_up[par], warps * ctas) == kGaveUp;  // the cluster agrees on giving up
    } else {
      if (lane == 0) sums[par][threadIdx.x >> 5] = dot;
      quit = team_any(team, T, !ok);  // so does the team
    }
    if (quit) break;
    // behind this barrier nobody reads the previous row's stage any more
    if (tid == 0 && ahead && next < p.rows) issue();
    ahead = true;
    if (CL) dot = join_sum<true>(sums[par], warps * ctas);
    else if (warps > 1) dot = join_sum<false>(sums[par] + team * warps, warps);
    const float mean = -rs * (dot * inv_cols);
    const float2 mean2 = make_float2(mean, mean);  // -mean(gw xh)
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const int v = it * T + tid;
      if (v < nv) {
        float2 g[VEC / 2], h[VEC / 2], d[VEC / 2];
        fetch(gs, v, g);
        fetch(hs, v, h);
        if (DRES) fetch(ds, v, d);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          const float2 xh = f2_mul(h[j], rs2);
          const float2 gw = f2_mul(g[j], w[it * (VEC / 2) + j]);
          dw[it * (VEC / 2) + j] = f2_fma(g[j], xh, dw[it * (VEC / 2) + j]);
          const float2 t = f2_fma(xh, mean2, gw);
          d[j] = DRES ? f2_fma(t, rs2, d[j]) : f2_mul(t, rs2);
        }
        const int c0 = col0 + v * VEC;
        const uint4 u = vec_narrow<XT>(reinterpret_cast<const float*>(d));
        char* to = static_cast<char*>(p.dx) + (row_at + c0) * elem_bytes<XT>();
        if (SHIFT && is_edge<VEC>(c0, p.cols)) store_edge_vec<XT>(to, c0, p.cols, u);
        else vec_store(to, u);
      }
    }
    if (++stage == stages) { stage = 0; phase ^= 1u; }
    par ^= 1;
    row = row_next;
  }
  if (quit && tid == 0) drain_stages(full[team], stages, stage, phase, next_stage);
  if (p.part == nullptr && !quit) return;
  if (__syncthreads_or(quit)) return;  // every team is through with its ring
  float* to = teams == 1 ? p.part + static_cast<int64_t>(unit) * p.cols
                         : reinterpret_cast<float*>(smem) + static_cast<int64_t>(team) * p.cols;
#pragma unroll
  for (int it = 0; it < ITEMS; ++it) {
    const int v = it * T + tid;
    if (SHIFT) {
      const float* f = reinterpret_cast<const float*>(dw + it * (VEC / 2));
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int c = col0 + v * VEC + j;
        if (v < nv && c >= 0 && c < p.cols) to[c] = f[j];
      }
    } else if (v < nv) {
#pragma unroll
      for (int j = 0; j < VEC / 2; j += 2) {
        const float2 a = dw[it * (VEC / 2) + j], b = dw[it * (VEC / 2) + j + 1];
        *reinterpret_cast<float4*>(to + col0 + v * VEC + 2 * j) = make_float4(a.x, a.y, b.x, b.y);
      }
    }
  }
  if (teams == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
    float t = 0.0f;
    for (int k = 0; k < teams; ++k) t += reinterpret_cast<const float*>(smem)[k * p.cols + c];
    p.part[static_cast<int64_t>(blockIdx.x) * p.cols + c] = t;
  }
}

// dweight[c] = sum of the partials of column c.  A CTA takes 32 columns, its
// warp w every W-th partial row from w, ten of them in flight at once; the
// warps' sums join in order.  32 warps (the norm's 296 partial rows in one go:
// 8 warps took 10 us, load latency) as long as one wave of CTAs holds all
// columns with them, else fewer, and no more than there are partial rows.
constexpr int kDwWarps = 32;
constexpr int kDwFlight = 10;
constexpr int64_t kDwThreads = 148 * 2048;  // a wave
__global__ void __launch_bounds__(32 * kDwWarps) k_column_partials(const float* part, int parts, int cols, void* out, int ot) {
  __shared__ float s[kDwWarps][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float acc = 0.0f;
  if (c < cols)
    for (int b0 = warp; b0 < parts; b0 += warps * kDwFlight) {
      float f[kDwFlight];
#pragma unroll
      for (int k = 0; k < kDwFlight; ++k) {
        const int b = b0 + k * warps;
        f[k] = b < parts ? __ldcg(part + static_cast<int64_t>(b) * cols + c) : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < kDwFlight; ++k) acc += f[k];
    }
  s[warp][lane] = acc;
  __syncthreads();
  // a column of the tile at a time: its warps' sums, joined over the lanes
  for (int cw = warp; cw < 32; cw += warps) {
    const float t = warp_sum(lane < warps ? s[lane][cw] : 0.0f);
    if (lane == 0 && blockIdx.x * 32 + cw < cols) elem_store_rt(out, ot, blockIdx.x * 32 + cw, t);
  }
}

int sm_count() {
  int dev = 0;
  cudaGetDevice(&dev);
  return device_sm_count(dev);
}

// Opens up to kRingSmem of dynamic shared memory to a ring kernel, once per
// device.
constexpr int kRingSmem = 224 * 1024;
template <typename K>
cudaError_t open_smem(K kernel, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int ring_threads(int64_t cols, int e) { return static_cast<int>(((cols + e - 1) / e + 31) / 32 * 32); }

// Elements per thread for rows of `cols`: the share that keeps the most of an
// SM's 512 threads busy (1408 columns of bf16, 47616 rows: 24 elements in 8
// CTAs of 64 threads 78 us, 16 elements in 4 of 96 threads 101 us), up to
// `most` elements unless fewer do not reach.  Of equals the widest for one
// tensor a row (what a row costs every warp, the joins and divisions, is
// shared by more elements: [16384, 8192] bf16 without a residual 97 us with
// 32, 126 with 16), else the narrowest (with one 171 and 145).
int ring_share(int64_t cols, int most, bool widest) {
  if (cols <= 256) return 8;
  int best = 0;
  double busy = 0.0;
  for (int e : {16, 24, 32}) {
    const int t = ring_threads(cols, e);
    if (t > ring_max_threads(e) || (e > most && best != 0)) continue;
    const double b = static_cast<double>(ring_max_threads(e) / t) * static_cast<double>(cols) / e;
    if (b > busy || (widest && b == busy)) { busy = b; best = e; }
  }
  return best;
}

// bytes of a row in a stage, and the columns that a row's vectors reach over
template <int XT, bool SHIFT>
int64_t stage_row(int64_t cols) {
  return SHIFT ? shifted_vecs<vec_elems<XT>()>(static_cast<int>(cols)) * 16ll : cols * elem_bytes<XT>();
}
template <int XT, bool SHIFT>
int64_t reach(int64_t cols) {
  return SHIFT ? shifted_vecs<vec_elems<XT>()>(static_cast<int>(cols)) * vec_elems<XT>() : cols;
}

// Shared memory of a CTA beside its stages.
constexpr int kNormSpare = 1024 + 1024, kBwdSpare = 2048 + 1024;
// Whether a row is more than a CTA's columns or two stages take.
template <int XT, bool SHIFT>
bool wide(int64_t cols, int tensors) {
  return reach<XT, SHIFT>(cols) > kRingMaxCols || 2 * stage_row<XT, SHIFT>(cols) * tensors > kRingSmem - kBwdSpare;
}
// A row has two whole vectors at least, wherever it starts.
template <int XT>
bool shift_fits(int64_t cols) {
  return cols >= 3 * vec_elems<XT>();
}

template <int XT, int E, bool RES, bool SHIFT>
cudaError_t norm_ring(const NormArgs& a, const NormParams& p) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = open_smem(k_rmsnorm_ring<XT, E, RES, SHIFT, false>, done);
  if (e != cudaSuccess) return e;
  const int64_t stage = stage_row<XT, SHIFT>(a.cols) * (RES ? 2 : 1);
  const int threads = ring_threads(reach<XT, SHIFT>(a.cols), E);
  // as many CTAs on an SM as the registers allow, while two stages each fit
  int ctas = ring_max_threads(E) / threads;
  if (ctas > 32) ctas = 32;
  while (ctas > 1 && (kRingSmem / ctas - kNormSpare) / stage < 2) --ctas;
  int64_t stages = (kRingSmem / ctas - kNormSpare) / stage;
  if (stages > kRingStages) stages = kRingStages;
  const int64_t most = static_cast<int64_t>(sm_count()) * ctas;
  // a CTA's rows start at one place of a vector: VEC rows apart, or one row
  const int64_t grid = row_grid(a.rows, most, SHIFT ? vec_elems<XT>() : 1);
  const int64_t per = (a.rows + grid - 1) / grid;
  if (stages > per) stages = per;
  return launch_pdl(k_rmsnorm_ring<XT, E, RES, SHIFT, false>, dim3(static_cast<unsigned>(grid)), dim3(threads),
                    static_cast<size_t>(stages * stage), a.stream, false, p, static_cast<int>(stages), device_error_word());
}

// How rows are split over a cluster: its CTAs, elements per thread and stages.
// Two CTAs where two stages fit and their threads hold no more than max_e
// elements, four for few rows ([32, 28672] bf16 3.9 us in four, 4.9 in two)
// and otherwise: the barrier's time counts per row ([4096, 20480] bf16 with a
// residual 139 us in two, 211 in four, 337 in eight).  max_e is 32, but 16 for
// the forward pass of f32 rows with a residual, whose vectors take the most
// registers ([4096, 24576]: 278 us in four CTAs, 326 in two with 24 elements).
// A CTA's share is wide enough that one runs on an SM.  tensors: rows that a
// stage holds; spare: shared memory of a CTA beside its stages.
struct ClusterPlan {
  int ctas, e, threads, stages;
  size_t smem;
};
template <int XT, bool SHIFT>
ClusterPlan cluster_plan(int64_t rows, int64_t cols, int tensors, int spare, int max_e) {
  ClusterPlan c{};
  for (c.ctas = 4 * rows <= sm_count() ? 4 : 2;; c.ctas *= 2) {
    const int share = cluster_share<vec_elems<XT>(), SHIFT>(static_cast<int>(cols), c.ctas);
    const int64_t stage = static_cast<int64_t>(share) * 16 * tensors;
    const int n = share * vec_elems<XT>();
    c.e = n <= 16 * 512 ? 16 : n <= 24 * 512 ? 24 : 32;
    c.threads = ring_threads(n, c.e);
    if (c.ctas < 4 && (c.threads > 512 || c.e > max_e || 2 * stage > kRingSmem - spare)) continue;
    c.stages = static_cast<int>((kRingSmem - spare) / stage);
    if (c.stages > kRingStages) c.stages = kRingStages;
    c.smem = static_cast<size_t>(c.stages * stage);
    return c;
  }
}

// The clusters of a plan that run at the same time; the last answer is kept
// (the same on every B200).
template <typename K>
int clusters_at_once(K kernel, const ClusterPlan& c, std::atomic<uint64_t>& last) {
  const uint64_t key = (static_cast<uint64_t>(c.smem) << 32) | (static_cast<uint64_t>(c.threads) << 20) | (c.ctas << 16);
  const uint64_t known = last.load(std::memory_order_acquire);
  if ((known & ~0xFFFFull) == key && (known & 0xFFFF) != 0) return static_cast<int>(known & 0xFFFF);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c.ctas * 16, 1, 1);
  cfg.blockDim = dim3(c.threads, 1, 1);
  cfg.dynamicSmemBytes = c.smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = c.ctas;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int fit = 0;
  if (cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) != cudaSuccess || fit < 1) {
    cudaGetLastError();
    fit = sm_count() / c.ctas;
  }
  last.store(key | static_cast<uint64_t>(fit), std::memory_order_release);
  return fit;
}

template <int XT, int E, bool RES, bool SHIFT>
cudaError_t norm_cluster(const NormArgs& a, const NormParams& p, const ClusterPlan& c) {
  static std::atomic<uint64_t> done{0}, last{0};
  const auto kernel = k_rmsnorm_ring<XT, E, RES, SHIFT, true>;
  const cudaError_t e = open_smem(kernel, done);
  if (e != cudaSuccess) return e;
  const int64_t grid = row_grid(a.rows, clusters_at_once(kernel, c, last), SHIFT ? vec_elems<XT>() : 1);
  return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(grid * c.ctas)), dim3(c.threads), c.smem, a.stream, c.ctas, p,
                            c.stages, device_error_word());
}

template <int XT, bool RES, bool SHIFT>
cudaError_t norm_ring_any(const NormArgs& a, const NormParams& p) {
  const int64_t cols = reach<XT, SHIFT>(a.cols);
  if (wide<XT, SHIFT>(a.cols, RES ? 2 : 1)) {
    const ClusterPlan c = cluster_plan<XT, SHIFT>(a.rows, a.cols, RES ? 2 : 1, kNormSpare, XT == 0 && RES ? 16 : 32);
    if (c.e == 32) return norm_cluster<XT, 32, RES, SHIFT>(a, p, c);
    return c.e == 16 ? norm_cluster<XT, 16, RES, SHIFT>(a, p, c) : norm_cluster<XT, 24, RES, SHIFT>(a, p, c);
  }
  if (a.rows <= sm_count() && cols <= 8 * 1024) return norm_ring<XT, 8, RES, SHIFT>(a, p);
  // the elements that fit the registers: fewer where rows share vectors, fewer
  // with a second tensor in f32 (8192 x 5001: 120 us with 16, 186 with 24)
  constexpr int kMost = !RES && !SHIFT ? 32 : RES && SHIFT && XT == 0 ? 16 : 24;
  switch (ring_share(cols, kMost, !RES)) {
    case 32: return norm_ring<XT, 32, RES, SHIFT>(a, p);
    case 24: return norm_ring<XT, 24, RES, SHIFT>(a, p);
    case 16: return norm_ring<XT, 16, RES, SHIFT>(a, p);
    default: return norm_ring<XT, 8, RES, SHIFT>(a, p);
  }
}

template <int XT>
cudaError_t norm_run(const NormArgs& a, const NormParams& p) {
  constexpr int VEC = vec_elems<XT>();
  const int group = p.block / VEC;
  const bool vecs = aligned16(a.x) && aligned16(a.residual) && aligned16(a.residual_out) && aligned16(a.y_out) &&
                    reinterpret_cast<uintptr_t>(a.q) % VEC == 0 &&
                    (p.block == 0 || (group <= 32 && (group & (group - 1)) == 0));
  if (vecs && a.cols % VEC == 0 && aligned16(a.weight))
    return a.residual ? norm_ring_any<XT, true, false>(a, p) : norm_ring_any<XT, false, false>(a, p);
  if (vecs && p.block == 0 && shift_fits<XT>(a.cols))
    return a.residual ? norm_ring_any<XT, true, true>(a, p) : norm_ring_any<XT, false, true>(a, p);
  const int64_t grid = a.rows < 8 * sm_count() ? a.rows : 8 * sm_count();
  return launch_pdl(k_rmsnorm_any<XT>, dim3(static_cast<unsigned>(grid)), dim3(kAnyThreads), 0, a.stream, false, p);
}

int64_t bwd_parts(int64_t rows) { return rows < kBwdParts ? rows : kBwdParts; }

template <int XT, int E, bool DRES, bool SHIFT>
cudaError_t bwd_cluster(const NormBwdArgs& a, const NormBwdParams& p, const ClusterPlan& c, int64_t& grid) {
  static std::atomic<uint64_t> done{0}, last{0};
  const auto kernel = k_rmsnorm_bwd_ring<XT, E, DRES, SHIFT, true>;
  const cudaError_t e = open_smem(kernel, done);
  if (e != cudaSuccess) return e;
  grid = row_grid(a.rows, clusters_at_once(kernel, c, last), SHIFT ? vec_elems<XT>() : 1);  // partial rows too
  return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(grid * c.ctas)), dim3(c.threads), c.smem, a.stream, c.ctas, p, 1,
                            c.stages, device_error_word());
}

template <int XT, int E, bool DRES, bool SHIFT>
cudaError_t bwd_ring(const NormBwdArgs& a, const NormBwdParams& p, int64_t& grid) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = open_smem(k_rmsnorm_bwd_ring<XT, E, DRES, SHIFT, false>, done);
  if (e != cudaSuccess) return e;
  const int64_t stage = stage_row<XT, SHIFT>(a.cols) * (DRES ? 3 : 2);
  const int T = ring_threads(reach<XT, SHIFT>(a.cols), E);
  const int half = ring_max_threads(E) / 2;
  // CTAs of half the threads that the registers allow, two to an SM, while
  // every team has a row
  int teams = half / T;
  if (teams > kTeams) teams = kTeams;
  const int64_t sms = sm_count();
  while (teams > 1 && (static_cast<int64_t>(teams) * sms >= 2 * a.rows || 2 * teams * stage > kRingSmem / 2 - kBwdSpare)) --teams;
  if (teams < 1) teams = 1;
  const int ctas = (T * teams <= half && 2 * teams * stage <= kRingSmem / 2 - kBwdSpare) ? 2 : 1;
  int64_t most = sms * ctas;
  if (most > kBwdParts) most = kBwdParts;
  // a team's rows start at one place of a vector: VEC rows apart, or one row
  grid = row_grid((a.rows + teams - 1) / teams, most, SHIFT ? vec_elems<XT>() : 1);
  const int64_t per = (a.rows + grid * teams - 1) / (grid * teams);
  int64_t stages = (kRingSmem / ctas - kBwdSpare) / (teams * stage);
  if (stages > kRingStages) stages = kRingStages;
  if (stages > per) stages = per;
  return launch_pdl(k_rmsnorm_bwd_ring<XT, E, DRES, SHIFT, false>, dim3(static_cast<unsigned>(grid)), dim3(T * teams),
                    static_cast<size_t>(stages * teams * stage), a.stream, false, p, teams, static_cast<int>(stages),
                    device_error_word());
}

template <int XT, bool DRES, bool SHIFT>
cudaError_t bwd_ring_any(const NormBwdArgs& a, const NormBwdParams& p, int64_t& grid) {
  const int64_t cols = reach<XT, SHIFT>(a.cols);
  if (wide<XT, SHIFT>(a.cols, DRES ? 3 : 2)) {
    const ClusterPlan c = cluster_plan<XT, SHIFT>(a.rows, a.cols, DRES ? 3 : 2, kBwdSpare, 32);
    if (c.e == 32) return bwd_cluster<XT, 32, DRES, SHIFT>(a, p, c, grid);
    return c.e == 16 ? bwd_cluster<XT, 16, DRES, SHIFT>(a, p, c, grid) : bwd_cluster<XT, 24, DRES, SHIFT>(a, p, c, grid);
  }
  switch (ring_share(cols, 24, false)) {
    case 32: return bwd_ring<XT, 32, DRES, SHIFT>(a, p, grid);
    case 24: return bwd_ring<XT, 24, DRES, SHIFT>(a, p, grid);
    case 16: return bwd_ring<XT, 16, DRES, SHIFT>(a, p, grid);
    default: return bwd_ring<XT, 8, DRES, SHIFT>(a, p, grid);
  }
}

// grid: the largest number of CTAs (and partial rows); the number launched.
template <int XT>
cudaError_t bwd_run(const NormBwdArgs& a, const NormBwdParams& p, int64_t& grid) {
  constexpr int VEC = vec_elems<XT>();
  const bool vecs = aligned16(a.dy) && aligned16(a.h) && aligned16(a.dres) && aligned16(a.dx);
  if (vecs && a.cols % VEC == 0 && aligned16(a.weight))
    return a.dres ? bwd_ring_any<XT, true, false>(a, p, grid) : bwd_ring_any<XT, false, false>(a, p, grid);
  if (vecs && shift_fits<XT>(a.cols))
    return a.dres ? bwd_ring_any<XT, true, true>(a, p, grid) : bwd_ring_any<XT, false, true>(a, p, grid);
  const size_t smem = p.part ? static_cast<size_t>(a.cols) * 4 : 0;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k_rmsnorm_bwd_any<XT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kNormMaxCols * 4));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k_rmsnorm_bwd_any<XT>, dim3(static_cast<unsigned>(grid)), dim3(kAnyThreads), smem, a.stream, false, p);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a) {
  NormParams p;
  p.x = a.x; p.residual = a.residual; p.weight = a.weight; p.wt = a.wt;
  p.rows = static_cast<int>(a.rows); p.cols = static_cast<int>(a.cols); p.eps = a.eps; p.fmt = a.fmt;
  // a block as wide as the row is the row: the same scale at the same place
  p.block = a.block >= a.cols ? 0 : static_cast<int>(a.block);
  p.nb = p.block ? static_cast<int>((a.cols + p.block - 1) / p.block) : 0;
  p.q = a.q; p.scales = a.scales; p.residual_out = a.residual_out; p.y_out = a.y_out; p.rstd_out = a.rstd_out;
  if (a.xt == 0) return norm_run<0>(a, p);
  if (a.xt == 1) return norm_run<1>(a, p);
  return norm_run<2>(a, p);
}

size_t rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  return static_cast<size_t>(bwd_parts(rows)) * static_cast<size_t>(cols) * 4;
}

cudaError_t launch_rmsnorm_backward(const NormBwdArgs& a) {
  NormBwdParams p;
  p.dy = a.dy; p.h = a.h; p.dres = a.dres; p.weight = a.weight; p.wt = a.wt; p.rstd = a.rstd;
  p.rows = static_cast<int>(a.rows); p.cols = static_cast<int>(a.cols); p.dx = a.dx;
  p.part = a.dweight ? a.ws : nullptr;
  int64_t parts = bwd_parts(a.rows);
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    if (a.xt == 0) e = bwd_run<0>(a, p, parts);
    else if (a.xt == 1) e = bwd_run<1>(a, p, parts);
    else e = bwd_run<2>(a, p, parts);
  }
  if (e != cudaSuccess || !a.dweight) return e;
  return launch_column_partials(a.ws, static_cast<int>(parts), p.cols, a.dweight, a.wt, a.stream);
}

cudaError_t launch_column_partials(const float* part, int parts, int cols, void* out, int ot, cudaStream_t stream) {
  const int64_t tiles = (static_cast<int64_t>(cols) + 31) / 32;
  int warps = kDwWarps;
  while (warps > 4 && (tiles * 32 * warps > kDwThreads || warps / 2 >= parts)) warps /= 2;
  return launch_pdl(k_column_partials, dim3(static_cast<unsigned>(tiles)), dim3(32 * warps), 0, stream, false, part, parts, cols,
                    out, ot);
}

}  // namespace hq
