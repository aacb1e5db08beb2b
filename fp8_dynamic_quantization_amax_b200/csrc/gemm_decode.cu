// gemm_decode.cu -- the activation GEMM for up to 16 rows and few columns
// (decode): out = bf16(act(acc x_scale w_scale + bias) + residual), split
// over K inside a thread-block cluster.  sm_100a only.
//
// One tcgen05.mma takes some 70 cycles however few columns it has (up to
// 128; M of 64 or 128 alike), so the 64-column tiles that spread N = 8192
// over 128 SMs spend 310 cycles of every 128-byte K block issuing four of
// them, more than the block's weight bytes take to arrive: 54 us at N = 8192,
// K = 28672, M = 1.  Here S CTAs (a cluster, S = 2, 4 or 8) share a tile of up
// to 128 columns, each a run of K: half the products or fewer per weight
// byte, and all SMs busy where N alone would not fill them.  Against those
// tiles, us: M = 1, N = 8192, K = 28672 42.7 and 54-61; M = 16, N = K = 8192
// 16.9 and 20.3; M = 4, N = K = 4096 7.8 and 11.5; M = 16, N = 1024, K = 4096
// 5.5 and 10.7; M = 8, N = 512, K = 8192 6.0 and 16.8.
//
// Warp 0 streams K slices of X (16 rows) and W through TMA, one lane of warp
// 1 issues the products into tensor memory, warp 4 puts the rows of the CTA's
// partial sums into shared memory.  After a cluster
// barrier every CTA finishes its share of the tile's columns: it adds the S
// partial sums in rank order (a fixed order) from the cluster's shared
// memories and applies scales, bias, activation and residual.
#include "act.cuh"
#include "hq_internal.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "tc.cuh"

#include <atomic>
#include <cstring>

namespace hq {
namespace {

constexpr int kDkRows = 16;                        // rows of X
constexpr int kDkCols = 128;                       // columns of a tile, at most
constexpr int kDkThreads = 6 * 32;                 // TMA, MMA, warp 4 reads the sums, all finish
constexpr int kDkStages = 5, kDkBlocks = 2;        // stages of kDkBlocks K blocks (3 x 3: 1 % slower, 2 x 5 and 10 x 1: 7-13 %)
constexpr int kDkA = kDkRows * kTcKBytes, kDkB = kDkCols * kTcKBytes;
constexpr int kDkPad = kDkCols + 4;                // floats per row of partial sums
constexpr int kDkSmem = kDkStages * kDkBlocks * (kDkA + kDkB) + 1024;
// the product reads 128 rows of A from a block's start: past the 16 loaded,
// what follows in shared memory, into accumulator rows that nothing reads
static_assert((kDkStages * kDkBlocks - 1) * kDkA + 128 * kTcKBytes <= kDkStages * kDkBlocks * (kDkA + kDkB), "reads stay inside");
static_assert(kDkRows * kDkPad * 4 + kDkSmem + 512 <= 232448, "shared memory over the 227 KB per-CTA limit");

struct DecodeParams {
  int M, N, nkb;
  int width;             // columns per tile, a multiple of 8
  uint32_t idesc;
  const float* xs;
  const float* ws;
  int xs_bcast, ws_bcast;
  const uint16_t* bias;
  const uint16_t* res;   // may be out itself
  uint16_t* out;
  int act;
  unsigned* err;
};

// a float at shared-memory address addr of CTA rank of the cluster
__device__ __forceinline__ float load_cluster(uint32_t addr, uint32_t rank) {
  float f;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(f)
               : "r"(addr), "r"(rank)
               : "memory");
  return f;
}

__device__ __forceinline__ float act_one(float z, int act) {
  const float2 v = make_float2(z, 0.0f);
  switch (act) {
    case kActRelu: return act_forward<kActRelu>(v).x;
    case kActGelu: return act_forward<kActGelu>(v).x;
    case kActGeluTanh: return act_forward<kActGeluTanh>(v).x;
    case kActSilu: return act_forward<kActSilu>(v).x;
    default: return z;
  }
}

template <int S>
__global__ void __cluster_dims__(S, 1, 1) __launch_bounds__(kDkThreads, 1)
    k_gemm_decode(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const DecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) float part[kDkRows * kDkPad];
  __shared__ __align__(8) uint64_t full_bar[kDkStages];
  __shared__ __align__(8) uint64_t empty_bar[kDkStages];
  __shared__ __align__(8) uint64_t done_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const uint32_t raw = ptx::smem_u32(smem_raw);
  uint8_t* sA = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  uint8_t* sB = sA + kDkStages * kDkBlocks * kDkA;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_rank();
  const int col0 = static_cast<int>(blockIdx.x / S) * p.width;
  const int k0 = static_cast<int>(static_cast<int64_t>(rank) * p.nkb / S);  // this CTA's K blocks
  const int k1 = static_cast<int>(static_cast<int64_t>(rank + 1) * p.nkb / S);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return ptx::mbar_wait_inline(bar, parity, &abort_flag, p.err, kDevErrTimeout);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < kDkStages; ++s) {
      ptx::mbar_init(&full_bar[s], 1);
      ptx::mbar_init(&empty_bar[s], 1);
    }
    ptx::mbar_init(&done_bar, 1);
    abort_flag = 0;
    ptx::fence_mbarrier_init();
  }
  // Global memory only behind this; tensor memory too: an allocation held while
  // waiting for the previous grid could keep that grid's CTAs from theirs.
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_u32(&tmem_slot)),
                 "r"(static_cast<uint32_t>(kDkCols))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t block_bytes = static_cast<uint32_t>(kDkA + p.width * kTcKBytes);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t filled = 0, parity = 0;  // per stage: a fill is under way or done, and its parity
      for (int kb = k0; kb < k1; kb += kDkBlocks) {
        if (!wait(&empty_bar[stage], phase ^ 1u)) break;
        const int n = min(kDkBlocks, k1 - kb);
        ptx::mbar_arrive_expect_tx(&full_bar[stage], n * block_bytes);
        for (int u = 0; u < n; ++u) {
          tma_load_2d(sA + (stage * kDkBlocks + u) * kDkA, &tm_a, &full_bar[stage], (kb + u) * kTcKBytes, 0);
          tma_load_2d(sB + (stage * kDkBlocks + u) * kDkB, &tm_b, &full_bar[stage], (kb + u) * kTcKBytes, col0);
        }
        filled |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == kDkStages) { stage = 0; phase ^= 1u; }
      }
      if (abort_flag) {  // what is in flight lands before the CTA leaves
        int dummy = 0;
        for (int s = 0; s < kDkStages; ++s)
          if (filled & (1u << s)) ptx::mbar_wait(&full_bar[s], (parity >> s) & 1u, &dummy, nullptr, 0, ptx::kDrainLimitNs);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool issued = false;
      for (int kb = k0; kb < k1; kb += kDkBlocks) {
        if (!wait(&full_bar[stage], phase)) break;
        tc_fence_after();
        const int n = min(kDkBlocks, k1 - kb);
        for (int u = 0; u < n; ++u) {
          const uint64_t ad = smem_desc(ptx::smem_u32(sA + (stage * kDkBlocks + u) * kDkA));
          const uint64_t bd = smem_desc(ptx::smem_u32(sB + (stage * kDkBlocks + u) * kDkB));
#pragma unroll
          for (int k = 0; k < kTcKBytes / 32; ++k)
            mma_issue<0>(tmem, ad + 2u * k, bd + 2u * k, p.idesc, (kb + u > k0 || k > 0) ? 1u : 0u);
        }
        tc_commit(&empty_bar[stage]);
        issued = true;
        if (++stage == kDkStages) { stage = 0; phase ^= 1u; }
      }
      // all products of this CTA; also what an aborted loop left in flight
      if (issued) tc_commit(&done_bar);
      else ptx::mbar_arrive(&done_bar);
      if (abort_flag) {
        int dummy = 0;
        ptx::mbar_wait(&done_bar, 0, &dummy, nullptr, 0, ptx::kDrainLimitNs);
      }
    }
    __syncwarp();
  } else {
    // rows 0 .. 15 of the accumulator are lanes 0 .. 15 of tensor-memory lane
    // quadrant 0, which only warps with index 0 mod 4 may read: warp 4 reads
    // every column
    if (warp == 4) {
      const bool ok = !__any_sync(0xFFFFFFFFu, !wait(&done_bar, 0));
      tc_fence_after();
      if (ok) {
        const bool any = k1 > k0;  // a run of no K blocks leaves the accumulator unwritten
#pragma unroll 1
        for (int c = 0; c < p.width; c += 32) {
          uint32_t v[32];
          tmem_ld32(tmem + static_cast<uint32_t>(c), v);
          if (lane < kDkRows) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4*>(&part[lane * kDkPad + c + j]) =
                  any ? make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]) : make_uint4(0, 0, 0, 0);
          }
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  ptx::cluster_barrier();  // every CTA's partial sums are in its shared memory
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(static_cast<uint32_t>(kDkCols))
                 : "memory");
  }
  if (!abort_flag) {
    // this CTA's share of the tile's columns, in pairs (N and width are even)
    const int cols = min(p.width, p.N - col0);
    const int pairs = cols / 2;
    const int c0 = static_cast<int>(rank) * pairs / S, c1 = (static_cast<int>(rank) + 1) * pairs / S;
    const uint32_t base = ptx::smem_u32(part);
    for (int i = threadIdx.x; i < p.M * (c1 - c0); i += kDkThreads) {
      const int m = i / (c1 - c0);
      const int c = 2 * (c0 + i - m * (c1 - c0));
      const int n = col0 + c;
      float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
      for (int r = 0; r < S; ++r) {
        a0 += load_cluster(base + static_cast<uint32_t>(m * kDkPad + c) * 4, r);
        a1 += load_cluster(base + static_cast<uint32_t>(m * kDkPad + c + 1) * 4, r);
      }
      const float xsv = __ldg(p.xs + (p.xs_bcast ? 0 : m));
      const float s0 = __ldg(p.ws + (p.ws_bcast ? 0 : n)) * xsv, s1 = __ldg(p.ws + (p.ws_bcast ? 0 : n + 1)) * xsv;
      uint32_t b = 0;
      if (p.bias) b = __ldg(reinterpret_cast<const uint32_t*>(p.bias + n));
      float z0 = act_one(fmaf(a0, s0, __uint_as_float(b << 16)), p.act);
      float z1 = act_one(fmaf(a1, s1, __uint_as_float(b & 0xFFFF0000u)), p.act);
      const int64_t at = static_cast<int64_t>(m) * p.N + n;
      if (p.res) {
        const uint32_t r = *reinterpret_cast<const volatile uint32_t*>(p.res + at);
        z0 += __uint_as_float(r << 16);
        z1 += __uint_as_float(r & 0xFFFF0000u);
      }
      *reinterpret_cast<uint32_t*>(p.out + at) = pack_bf16x2(z0, z1);
    }
  }
  ptx::cluster_barrier();  // no CTA leaves while another may still read its sums
}

template <int S>
cudaError_t setup(int dev, int* clusters) {
  static std::atomic<int> known[64];  // 1 + the clusters that fit, by device
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int n = known[dev].load(std::memory_order_acquire);
  if (n == 0) {
    cudaError_t e = cudaFuncSetAttribute(k_gemm_decode<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDkSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S * 16, 1, 1);
    cfg.blockDim = dim3(kDkThreads, 1, 1);
    cfg.dynamicSmemBytes = kDkSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = S;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, k_gemm_decode<S>, &cfg) != cudaSuccess || fit < 1) {
      cudaGetLastError();
      fit = device_sm_count(dev) / S;
    }
    n = fit + 1;
    known[dev].store(n, std::memory_order_release);
  }
  *clusters = n - 1;
  return cudaSuccess;
}

template <int S>
cudaError_t run(const GemmArgs& a, int clusters, std::string* msg) {
  int width = static_cast<int>(((a.N + clusters - 1) / clusters + 7) / 8 * 8);
  if (width < 16) width = 16;
  CUtensorMap ta, tb;
  memset(&ta, 0, sizeof(ta));
  memset(&tb, 0, sizeof(tb));
  if (a.K > 0 && (!make_map(&ta, a.a, static_cast<uint64_t>(a.M), static_cast<uint64_t>(a.K), 1, kDkRows, msg) ||
                  !make_map(&tb, a.b, static_cast<uint64_t>(a.N), static_cast<uint64_t>(a.K), 1,
                            static_cast<uint32_t>(width), msg)))
    return cudaErrorInvalidValue;
  DecodeParams p;
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.nkb = static_cast<int>((a.K + kTcKBytes - 1) / kTcKBytes);
  p.width = width;
  const uint32_t fmt = static_cast<uint32_t>(a.fmt);
  p.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(kDkCols >> 3) << 17) |
            (static_cast<uint32_t>(128 >> 4) << 24);  // f32 sums, E4M3 / E5M2, N = 128, M = 128
  p.xs = a.x_scale;
  p.xs_bcast = a.x_scale_len == 1;
  p.ws = a.w_scale;
  p.ws_bcast = a.w_scale_len == 1;
  p.bias = static_cast<const uint16_t*>(a.bias);
  p.res = static_cast<const uint16_t*>(a.residual);
  p.out = static_cast<uint16_t*>(a.out);
  p.act = a.act;
  p.err = device_error_word();
  const unsigned tiles = static_cast<unsigned>((a.N + width - 1) / width);
  return launch_pdl(k_gemm_decode<S>, dim3(tiles * S), dim3(kDkThreads), kDkSmem, a.stream, false, ta, tb, p);
}

}  // namespace

bool gemm_decode_takes(const GemmArgs& a) {
  // N up to 128 columns for each of the clusters of two that fit on the SMs;
  // beyond, a tile per SM has its 128 columns without a split
  int dev = 0, clusters = 0;
  if (a.M > kDkRows || a.z_q != nullptr || cudaGetDevice(&dev) != cudaSuccess) return false;
  return setup<2>(dev, &clusters) == cudaSuccess && a.N <= static_cast<int64_t>(clusters) * kDkCols;
}

cudaError_t launch_gemm_decode(const GemmArgs& a, std::string* msg) {
  int dev = 0, clusters = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // the most CTAs per tile at which a tile keeps within 128 columns
  e = setup<8>(dev, &clusters);
  if (e != cudaSuccess) return e;
  if (a.N <= static_cast<int64_t>(clusters) * kDkCols) return run<8>(a, clusters, msg);
  e = setup<4>(dev, &clusters);
  if (e != cudaSuccess) return e;
  if (a.N <= static_cast<int64_t>(clusters) * kDkCols) return run<4>(a, clusters, msg);
  e = setup<2>(dev, &clusters);
  if (e != cudaSuccess) return e;
  return run<2>(a, clusters, msg);
}

}  // namespace hq
