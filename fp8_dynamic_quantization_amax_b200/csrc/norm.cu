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
#include "elem.cuh"
#include "fp8_cvt.cuh"
#include "hq_internal.cuh"
#include "launch.cuh"

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
// third time when it holds an infinity or NaN): any alignment and width.
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

// dweight[c] = sum of the partials of column c.  A CTA takes 32 columns, its
// warp w the w-th eighth of the partial rows; the eighths join in order.
constexpr int kDwWarps = 8;
__global__ void __launch_bounds__(32 * kDwWarps) k_column_partials(const float* part, int parts, int cols, void* out, int ot) {
  __shared__ float s[kDwWarps][32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int per = (parts + kDwWarps - 1) / kDwWarps;
  const int b0 = min(parts, warp * per), b1 = min(parts, b0 + per);
  float acc = 0.0f;
  if (c < cols)
#pragma unroll 8
    for (int b = b0; b < b1; ++b) acc += __ldcg(part + static_cast<int64_t>(b) * cols + c);
  s[warp][lane] = acc;
  __syncthreads();
  if (warp == 0 && c < cols) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kDwWarps; ++w) t += s[w][lane];
    elem_store_rt(out, ot, c, t);
  }
}

int sm_count() {
  int dev = 0;
  cudaGetDevice(&dev);
  return device_sm_count(dev);
}

template <int XT>
cudaError_t norm_run(const NormArgs& a, const NormParams& p) {
  const int64_t grid = a.rows < 8 * sm_count() ? a.rows : 8 * sm_count();
  return launch_pdl(k_rmsnorm_any<XT>, dim3(static_cast<unsigned>(grid)), dim3(kAnyThreads), 0, a.stream, false, p);
}

int64_t bwd_parts(int64_t rows) { return rows < kBwdParts ? rows : kBwdParts; }

template <int XT>
cudaError_t bwd_run(const NormBwdArgs& a, const NormBwdParams& p, int64_t grid) {
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
  // a block wider than the row is the row
  p.block = static_cast<int>(a.block);
  p.nb = a.block ? static_cast<int>((a.cols + a.block - 1) / a.block) : 0;
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
  const int64_t parts = bwd_parts(a.rows);
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
  return launch_pdl(k_column_partials, dim3(static_cast<unsigned>((static_cast<int64_t>(cols) + 31) / 32)), dim3(32 * kDwWarps), 0, stream,
                    false, part, parts, cols, out, ot);
}

}  // namespace hq
