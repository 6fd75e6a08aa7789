// What the paged-attention kernels share: their arguments, the output helpers and the
// kernel that joins partial results.
#pragma once

#include <cuda_bf16.h>
#include <math.h>

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

// The kernel for few rows (bf16, d = 64 or 128): 16 mt rows a unit, mt = 1 or 2.
int paged_mma_grid();
size_t paged_mma_part_bytes(int mt, int d);
int paged_mma_requests();  // requests a launch takes
cudaError_t launch_paged_mma(AttnArgs a, int mt, int d, cudaStream_t stream);

// The tensor-core kernel for chunks of new tokens (bf16, d = 64 or 128): partial-result
// bytes for a grid, and its launch (a.part_o set; a.part_ml is placed behind it).
size_t paged_tc_part_bytes(int grid, int d);
int paged_tc_requests();
cudaError_t launch_paged_tc(AttnArgs a, int d, int grid, cudaStream_t stream);

namespace {

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
constexpr int kJoinRows = 8;  // rows a CTA joins, a warp each

// Joins the partial results of the units that share boundaries cut: CTA (c - 1, y) looks
// at the boundary between shares c - 1 and c, and if it is the first one inside its unit,
// joins rows y * 8 .. y * 8 + 7 of it over every share that holds a part.
template <int D, typename SCHED, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const AttnArgs a, int grid) {
  constexpr int M = SCHED::kM;
  __shared__ typename SCHED::Mem mem;
  SCHED sched;
  sched.template init<kJoinThreads>(a.s, &mem, 0, grid);
  const int c = blockIdx.x + 1;
  if (c >= sched.G) return;
  const long long b = sched.share(c), before = sched.share(c - 1);
  if (b >= sched.total) return;
  sched.locate(b);
  const long long u0 = sched.unit0;
  if (u0 == b || before > u0) return;
  int lo;
  bool empty;
  const long long u1 = u0 + sched.tiles(sched.r, sched.blk, &lo, &empty);
  int last = c;  // the last share that holds a part
  while (last + 1 < sched.G && sched.share(last + 1) < u1) ++last;

  const int lane = threadIdx.x & 31;
  const int rr = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
  const int row = sched.blk * M + rr;
  if (row >= sched.r.rows) return;
  const int slot0 = 2 * (c - 1) + (u0 > before ? 1 : 0);
  // part 0 is in slot0, part i in slot 2 (c - 1 + i)
  const int parts = last - c + 2;
  float m = -INFINITY;
  for (int i = lane; i < parts; i += 32)
    m = fmaxf(m, a.part_ml[(size_t)(i == 0 ? slot0 : 2 * (c - 1 + i)) * M + rr].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float safe = m == -INFINITY ? 0.f : m;
  constexpr int NL = (D + 31) / 32;  // columns a lane
  float acc[NL], l = 0.f;
#pragma unroll
  for (int j = 0; j < NL; ++j) acc[j] = 0.f;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const size_t at = (size_t)(i == 0 ? slot0 : 2 * (c - 1 + i)) * M + rr;
    const float2 ml = a.part_ml[at];
    const float w = exp2f(ml.x - safe);
    l = fmaf(w, ml.y, l);
#pragma unroll
    for (int j = 0; j < NL; ++j)
      if (lane + 32 * j < D) acc[j] = fmaf(w, a.part_o[at * D + lane + 32 * j], acc[j]);
  }
  const int tok = sched.r.q0 + row / a.s.g, head = sched.h * a.s.g + row % a.s.g;
  const size_t at = (size_t)tok * a.Hq + head;
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  if (a.lse && lane == 0) a.lse[at] = lse_of(m, l);
#pragma unroll
  for (int j = 0; j < NL; ++j)
    if (lane + 32 * j < D) st_out<BF16>(a.out, at * D + lane + 32 * j, acc[j] * inv);
}

template <int D, typename SCHED>
cudaError_t launch_join(const AttnArgs& a, bool bf16, int grid, cudaStream_t stream) {
  if (grid < 2) return cudaSuccess;
  const dim3 g(grid - 1, SCHED::kM / kJoinRows);
  if (bf16)
    paged_join_kernel<D, SCHED, true><<<g, kJoinThreads, 0, stream>>>(a, grid);
  else
    paged_join_kernel<D, SCHED, false><<<g, kJoinThreads, 0, stream>>>(a, grid);
  return cudaGetLastError();
}

}  // namespace
}  // namespace gdn
