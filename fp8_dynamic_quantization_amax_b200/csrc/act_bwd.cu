// act_bwd.cu -- backward pass of an activation from its 8-bit checkpoint,
// with the bias gradient: z = dec(z_q) * scale, dz = g * act'(z),
// dbias = column sums of dz.  sm_100a only.
//
// One pass over the data.  A CTA takes a strip of 256 columns (a warp's 32
// lanes x 8 columns) and a band of rows; warp w of the CTA takes rows w,
// w + 8, ... of the band, four rows' loads in flight.  With dbias each lane
// adds its columns' f32 dz in row order, the eight warps join in order, and
// the band's sums go to the workspace; a second launch adds the bands in
// order.  The order of the sums is fixed, and the workspace needs no initial
// state.
//
// Bound: memory, as long as the derivative keeps up (act.cuh says how); four
// CTAs of 256 threads on an SM hold the loads that this takes.  [16384, 28672]
// with dbias, erf GELU: bf16 399 us replayed from a graph, 472 in calls among
// others at the capped clock, 6.0 and 5.1 TB/s (one row in flight and erff:
// 571 us); f32 902-918 us, 4.7 TB/s (64 registers spill 52-84 bytes there).
// [2047, 4096] f16, SiLU: 8.4 us.
#include "act.cuh"
#include "elem.cuh"
#include "hq_internal.cuh"
#include "launch.cuh"

#include <cuda_fp16.h>

namespace hq {
namespace {

constexpr int kAbWarps = 8;
constexpr int kAbVec = 8;                    // columns per lane
constexpr int kAbStrip = 32 * kAbVec;        // columns per strip
constexpr int kAbRows = 4;                   // a warp's rows in flight
constexpr int64_t kAbMinBand = kAbWarps * kAbRows;  // rows per band, at least
constexpr int64_t kAbCtas = 16 * 148;        // aim: this many CTAs

__host__ __device__ inline int64_t ab_strips(int64_t cols) { return (cols + kAbStrip - 1) / kAbStrip; }
inline int64_t ab_band_rows(int64_t rows, int64_t cols) {
  const int64_t bands = (kAbCtas + ab_strips(cols) - 1) / ab_strips(cols);
  const int64_t r = (rows + bands - 1) / bands;
  return r < kAbMinBand ? kAbMinBand : r;
}
inline int64_t ab_bands(int64_t rows, int64_t cols) {
  const int64_t r = ab_band_rows(rows, cols);
  return (rows + r - 1) / r;
}

struct AbParams {
  const void* g;
  const uint8_t* zq;
  const float* zs;
  int64_t rows;
  int cols, block, nb;
  int64_t band_rows;
  int strips;
  void* dz;
  float* part;   // [bands, cols] or null
};

// two FP8 codes (low byte first) -> two f32, exact (every code is an f16)
template <int FMT>
__device__ __forceinline__ float2 decode2(uint32_t c2) {
  uint32_t h;
  const unsigned short s = static_cast<unsigned short>(c2);
  if (FMT == 0) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(s));
  else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(s));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <int GT, int FMT, int ACT>
__global__ void __launch_bounds__(32 * kAbWarps, 4) k_act_bwd(const AbParams p) {
  constexpr int GV = GT == 0 ? 2 : 1;  // 16-byte vectors of g per lane and row
  __shared__ float red[kAbWarps][kAbStrip];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int strip = static_cast<int>(blockIdx.x % p.strips);
  const int64_t band = blockIdx.x / p.strips;
  const int c0 = strip * kAbStrip + lane * kAbVec;
  const int64_t r0 = band * p.band_rows;
  const int64_t r1 = min(p.rows, r0 + p.band_rows);
  float2 acc[kAbVec / 2];
#pragma unroll
  for (int j = 0; j < kAbVec / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
  if (c0 < p.cols) {  // cols % 16 == 0: a lane's 8 columns are all inside
    const float* zs = p.zs + c0 / p.block;
    for (int64_t r = r0 + warp; r < r1; r += kAbWarps * kAbRows) {
      uint4 gr[kAbRows][GV];
      uint2 zc[kAbRows];
      float sc[kAbRows];
#pragma unroll
      for (int k = 0; k < kAbRows; ++k) {
        const int64_t row = r + k * kAbWarps;
        if (row < r1) {
          const int64_t i = row * p.cols + c0;
          const char* gp = static_cast<const char*>(p.g) + i * elem_bytes<GT>();
#pragma unroll
          for (int v = 0; v < GV; ++v) gr[k][v] = vec_load(gp + 16 * v);
          zc[k] = __ldg(reinterpret_cast<const uint2*>(p.zq + i));
          sc[k] = __ldg(zs + row * p.nb);
        }
      }
#pragma unroll
      for (int k = 0; k < kAbRows; ++k) {
        const int64_t row = r + k * kAbWarps;
        if (row < r1) {
          float2 g[kAbVec / 2], d[kAbVec / 2];
#pragma unroll
          for (int v = 0; v < GV; ++v) vec_widen<GT>(gr[k][v], reinterpret_cast<float*>(g) + 4 * v);
#pragma unroll
          for (int j = 0; j < kAbVec / 2; ++j) {
            const float2 z = f2_mul(decode2<FMT>((j < 2 ? zc[k].x : zc[k].y) >> (16 * (j & 1))), act_both(sc[k]));
            d[j] = f2_mul(g[j], act_backward<ACT, GT == 0>(z));
            acc[j] = f2_add(acc[j], d[j]);
          }
          char* dp = static_cast<char*>(p.dz) + (row * p.cols + c0) * elem_bytes<GT>();
#pragma unroll
          for (int v = 0; v < GV; ++v) vec_store(dp + 16 * v, vec_narrow<GT>(reinterpret_cast<const float*>(d) + 4 * v));
        }
      }
    }
  }
  if (p.part == nullptr) return;
#pragma unroll
  for (int j = 0; j < kAbVec / 2; j += 2)
    *reinterpret_cast<float4*>(&red[warp][lane * kAbVec + 2 * j]) = make_float4(acc[j].x, acc[j].y, acc[j + 1].x, acc[j + 1].y);
  __syncthreads();
  const int c = strip * kAbStrip + static_cast<int>(threadIdx.x);
  if (c < p.cols) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kAbWarps; ++w) t += red[w][threadIdx.x];
    p.part[band * p.cols + c] = t;
  }
}

template <int GT, int FMT>
cudaError_t ab_run(const ActBwdArgs& a, const AbParams& p, unsigned grid) {
  const dim3 b(32 * kAbWarps);
  switch (a.act) {
    case kActRelu: return launch_pdl(k_act_bwd<GT, FMT, kActRelu>, dim3(grid), b, 0, a.stream, false, p);
    case kActGelu: return launch_pdl(k_act_bwd<GT, FMT, kActGelu>, dim3(grid), b, 0, a.stream, false, p);
    case kActGeluTanh: return launch_pdl(k_act_bwd<GT, FMT, kActGeluTanh>, dim3(grid), b, 0, a.stream, false, p);
    default: return launch_pdl(k_act_bwd<GT, FMT, kActSilu>, dim3(grid), b, 0, a.stream, false, p);
  }
}

}  // namespace

size_t act_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return 0;
  return static_cast<size_t>(ab_bands(rows, cols)) * static_cast<size_t>(cols) * 4;
}

cudaError_t launch_act_backward(const ActBwdArgs& a) {
  AbParams p;
  p.g = a.g; p.zq = a.z_q; p.zs = a.z_scales; p.rows = a.rows; p.cols = static_cast<int>(a.cols);
  p.block = static_cast<int>(a.block);
  p.nb = static_cast<int>((a.cols + a.block - 1) / a.block);
  p.strips = static_cast<int>(ab_strips(a.cols));
  p.dz = a.dz;
  p.part = a.dbias ? a.ws : nullptr;
  int64_t bands = 0;
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    p.band_rows = ab_band_rows(a.rows, a.cols);
    bands = ab_bands(a.rows, a.cols);
    const unsigned grid = static_cast<unsigned>(p.strips * bands);
    if (a.gt == 0) e = a.fmt == 0 ? ab_run<0, 0>(a, p, grid) : ab_run<0, 1>(a, p, grid);
    else if (a.gt == 1) e = a.fmt == 0 ? ab_run<1, 0>(a, p, grid) : ab_run<1, 1>(a, p, grid);
    else e = a.fmt == 0 ? ab_run<2, 0>(a, p, grid) : ab_run<2, 1>(a, p, grid);
  }
  if (e != cudaSuccess || !a.dbias) return e;
  return launch_column_partials(a.ws, static_cast<int>(bands), p.cols, a.dbias, a.gt, a.stream);
}

}  // namespace hq
