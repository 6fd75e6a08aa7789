// What the paged-attention kernels share: their arguments, the output helpers and the
// kernel that joins partial results.
#pragma once

#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "paged_sched.cuh"

namespace gdn {

struct AttnArgs {
  const void* q;
  const void* kc;
  const void* vc;
  void* out;
  float* lse;      // may be null
  float* part_o;   // [2 CTAs][M][D] unnormalised sums
  float2* part_ml; // [2 CTAs][M] running maximum (log2 units) and sum
  long long q_stride;
  int Hq, bs, num_blocks;
  float scale_log2;
  SchedArgs s;
};

// The kernel for few rows (bf16, d = 64 or 128), 16 a unit: partial-result bytes, the
// requests a launch takes, and the launch (a.part_o set).
size_t paged_mma_part_bytes(int d);
int paged_mma_requests();
cudaError_t launch_paged_mma(AttnArgs a, int d, cudaStream_t stream);

// The same of the tensor-core kernel for chunks of new tokens (bf16, d = 64 or 128).
size_t paged_tc_part_bytes(int grid, int d);
int paged_tc_requests();
cudaError_t launch_paged_tc(AttnArgs a, int d, int grid, cudaStream_t stream);

namespace {

// A kernel launched to overlap the end of the one before it: wait for that one's results
// (before), and let the next one start (in the one before).
__device__ __forceinline__ void after_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_kernel_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float lse_of(float m, float l) {
  return m == -INFINITY ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
}
template <bool BF16>
__device__ __forceinline__ void st_out(void* p, size_t i, float x) {
  if (BF16)
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else
    reinterpret_cast<float*>(p)[i] = x;
}

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

// Joins the partial results of the units that share boundaries cut.  CTA (c - 1, y) looks at
// the boundary between shares c - 1 and c; the CTAs of all boundaries inside one unit share
// its rows.  A row of up to kJoinWarps parts takes a warp, one of more parts the whole CTA,
// a warp for every kJoinWarps-th part.  The parts are summed in the order of the shares, the
// warps in theirs: the same sums every time.
template <int D, typename SCHED, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ AttnArgs a, int grid) {
  constexpr int M = SCHED::kM;
  constexpr int NL = (D + 31) / 32;  // columns a lane
  __shared__ typename SCHED::Mem mem;
  __shared__ float acc_s[kJoinWarps][D], l_s[kJoinWarps];
  SCHED sched;
  sched.template init<kJoinThreads>(a.s, &mem, 0, grid);
  after_previous_kernel();
  const int c = blockIdx.x + 1;
  if (c >= sched.G) return;
  const long long b = sched.share(c);
  if (b >= sched.total) return;
  sched.locate(b);
  const long long u0 = sched.unit0;
  if (u0 == b) return;
  int lo;
  bool empty;
  const long long u1 = u0 + sched.tiles(sched.r, sched.blk, &lo, &empty);
  const int c0 = sched.share_of(u0), c1 = sched.share_of(u1 - 1);  // the shares that hold a part
  // part 0 is in slot0, part i in slot 2 (c0 + i)
  const int parts = c1 - c0 + 1, slot0 = 2 * c0 + (u0 > sched.share(c0) ? 1 : 0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = min(sched.r.rows - sched.blk * M, M);
  const int me = (c - 1 - c0) * gridDim.y + blockIdx.y, team = (parts - 1) * gridDim.y;
  const bool whole_cta = parts > kJoinWarps;
  const int row_step = whole_cta ? team : team * kJoinWarps;
  for (int rr = whole_cta ? me : me * kJoinWarps + warp; rr < rows; rr += row_step) {
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32)
      m = fmaxf(m, a.part_ml[(size_t)(i == 0 ? slot0 : 2 * (c0 + i)) * M + rr].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float safe = m == -INFINITY ? 0.f : m;
    float acc[NL], l = 0.f;
#pragma unroll
    for (int j = 0; j < NL; ++j) acc[j] = 0.f;
#pragma unroll 4
    for (int i = whole_cta ? warp : 0; i < parts; i += whole_cta ? kJoinWarps : 1) {
      const size_t at = (size_t)(i == 0 ? slot0 : 2 * (c0 + i)) * M + rr;
      const float2 ml = a.part_ml[at];
      const float w = exp2f(ml.x - safe);
      l = fmaf(w, ml.y, l);
#pragma unroll
      for (int j = 0; j < NL; ++j)
        if (lane + 32 * j < D) acc[j] = fmaf(w, a.part_o[at * D + lane + 32 * j], acc[j]);
    }
    if (whole_cta) {
#pragma unroll
      for (int j = 0; j < NL; ++j)
        if (lane + 32 * j < D) acc_s[warp][lane + 32 * j] = acc[j];
      if (lane == 0) l_s[warp] = l;
      __syncthreads();
      if (warp == 0) {
        for (int w = 1; w < kJoinWarps; ++w) {
          l += l_s[w];
#pragma unroll
          for (int j = 0; j < NL; ++j)
            if (lane + 32 * j < D) acc[j] += acc_s[w][lane + 32 * j];
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const int row = sched.blk * M + rr, t = a.s.by_g.div(row);
    const size_t at = (size_t)(sched.r.q0 + t) * a.Hq + sched.h * a.s.g + (row - t * a.s.g);
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    if (a.lse && lane == 0) a.lse[at] = lse_of(m, l);
#pragma unroll
    for (int j = 0; j < NL; ++j)
      if (lane + 32 * j < D) st_out<BF16>(a.out, at * D + lane + 32 * j, acc[j] * inv);
  }
}

// Queued behind the kernel that leaves the parts so that it starts, and reads the schedule,
// while that one ends (it waits for it before it reads a part).
template <int D, typename SCHED>
cudaError_t launch_join(const AttnArgs& a, bool bf16, int grid, cudaStream_t stream) {
  if (grid < 2) return cudaSuccess;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid - 1, std::max(1, SCHED::kM / 32));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, paged_join_kernel<D, SCHED, true>, a, grid)
              : cudaLaunchKernelEx(&cfg, paged_join_kernel<D, SCHED, false>, a, grid);
}

}  // namespace
}  // namespace gdn
