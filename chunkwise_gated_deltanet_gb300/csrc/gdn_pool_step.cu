// The gated delta rule over a few new tokens per request, on a pool of states
// (gdn_recurrent_step): for request n with tokens cu[n] .. cu[n+1] and state
// S = pool[state_index[n]], for every token in order and every value head h
//
//     p = S k,  u = beta (v - alpha p),  S <- alpha S + u k^T,  o = S q
//
// (Nyysyyan, "Gated-DeltaNet" section, first equation block), with key head
// h / (H / Hk).  The state is read once and written once however many tokens there are.
//
// For a token or two this is bound by HBM (8 dk dv bytes a (request, head)); the
// arithmetic, 8 dk dv operations a token on the CUDA cores, passes it at about a dozen
// tokens.  A row of S is independent of the others once k, q, alpha and beta are known,
// so a warp owns 8 rows: 4 lanes a row, each holding a quarter of the row's columns in
// registers for the whole call.  Four lanes (not a whole warp) a row keep the reductions
// at two shuffles a value; each lane's columns are every fourth float4, so that a warp's
// access covers 64 consecutive bytes of each of its rows.  The CTA's 4 warps (32 rows)
// share k and q, which they stage as fp32 in shared memory kStage tokens at a time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kStepThreads = 128;
constexpr int kLanes = 4;                             // lanes a row
constexpr int kRowsCta = kStepThreads / kLanes;       // 32
constexpr int kStage = 8;                             // tokens staged at a time

template <bool BF16>
__device__ __forceinline__ float ldf(const void* p, size_t i) {
  if (BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
  return reinterpret_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void stf(void* p, size_t i, float x) {
  if (BF16)
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else
    reinterpret_cast<float*>(p)[i] = x;
}

template <int DK, bool BF16>
__global__ void __launch_bounds__(kStepThreads) pool_step_kernel(const StepArgs a, int splits) {
  constexpr int NV = DK / 4 / kLanes;  // float4 of S a lane
  __shared__ __align__(16) float ks[kStage][DK];
  __shared__ __align__(16) float qs[kStage][DK];
  __shared__ float as[kStage], bs[kStage], kqs[kStage];

  const int unit = blockIdx.x / splits, row_blk = blockIdx.x - unit * splits;
  const int n = unit / a.H, h = unit - n * a.H, hk = h / (a.H / a.Hk);
  const int t0 = min(max(__ldg(a.cu_seqlens + n), 0), a.T);
  const int t1 = min(max(__ldg(a.cu_seqlens + n + 1), t0), a.T);
  if (t0 == t1) return;  // no tokens: the state stays as it is
  const int slot = __ldg(a.state_index + n);
  const int tid = threadIdx.x, sub = tid % kLanes;
  const int r = row_blk * kRowsCta + tid / kLanes;
  const bool live = r < a.dv;
  if (slot < 0 || slot >= a.slots) {  // no state: the outputs are zeros
    for (int t = t0; t < t1; ++t)
      if (live && sub == 0) stf<BF16>(a.out, ((size_t)t * a.H + h) * a.dv + r, 0.f);
    return;
  }
  const bool fresh = a.context_lens != nullptr && __ldg(a.context_lens + n) <= 0;
  float4* Sp = reinterpret_cast<float4*>(a.pool + (((size_t)slot * a.H + h) * a.dv + (live ? r : 0)) * DK);
  float4 s[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    s[i] = live && !fresh ? Sp[sub + kLanes * i] : make_float4(0.f, 0.f, 0.f, 0.f);

  for (int tb = t0; tb < t1; tb += kStage) {
    const int nt = min(kStage, t1 - tb);
    if (tb > t0) __syncthreads();  // the last stage's readers are done
    for (int e = tid; e < nt * DK; e += kStepThreads) {
      const int j = e / DK, c = e - j * DK;
      ks[j][c] = ldf<BF16>(a.k, (size_t)(tb + j) * a.k_stride + (size_t)hk * DK + c);
      qs[j][c] = ldf<BF16>(a.q, (size_t)(tb + j) * a.q_stride + (size_t)hk * DK + c);
    }
    if (tid < nt) {
      as[tid] = expf(__ldg(a.log_alpha + (size_t)(tb + tid) * a.H + h));
      bs[tid] = __ldg(a.beta + (size_t)(tb + tid) * a.H + h);
    }
    __syncthreads();
    // k . q of each staged token, a warp a token
    for (int j = tid >> 5; j < nt; j += kStepThreads / 32) {
      float x = 0.f;
      for (int c = tid & 31; c < DK; c += 32) x = fmaf(ks[j][c], qs[j][c], x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if ((tid & 31) == 0) kqs[j] = x;
    }
    __syncthreads();
    for (int j = 0; j < nt; ++j) {
      const size_t at = ((size_t)(tb + j) * a.H + h) * a.dv + r;
      const float vr = live ? ldf<BF16>(a.v, (size_t)(tb + j) * a.v_stride + (size_t)h * a.dv + r) : 0.f;
      const float al = as[j];
      float p = 0.f, sq = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float4 kk = *reinterpret_cast<const float4*>(&ks[j][4 * (sub + kLanes * i)]);
        const float4 qq = *reinterpret_cast<const float4*>(&qs[j][4 * (sub + kLanes * i)]);
        p = fmaf(s[i].x, kk.x, p); p = fmaf(s[i].y, kk.y, p);
        p = fmaf(s[i].z, kk.z, p); p = fmaf(s[i].w, kk.w, p);
        sq = fmaf(s[i].x, qq.x, sq); sq = fmaf(s[i].y, qq.y, sq);
        sq = fmaf(s[i].z, qq.z, sq); sq = fmaf(s[i].w, qq.w, sq);
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) {
        p += __shfl_xor_sync(0xffffffffu, p, o);
        sq += __shfl_xor_sync(0xffffffffu, sq, o);
      }
      const float u = bs[j] * (vr - al * p);
      if (live && sub == 0) stf<BF16>(a.out, at, fmaf(al, sq, u * kqs[j]));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float4 kk = *reinterpret_cast<const float4*>(&ks[j][4 * (sub + kLanes * i)]);
        s[i].x = fmaf(al, s[i].x, u * kk.x);
        s[i].y = fmaf(al, s[i].y, u * kk.y);
        s[i].z = fmaf(al, s[i].z, u * kk.z);
        s[i].w = fmaf(al, s[i].w, u * kk.w);
      }
    }
  }
  if (live) {
#pragma unroll
    for (int i = 0; i < NV; ++i) Sp[sub + kLanes * i] = s[i];
  }
}

template <int DK>
cudaError_t launch_dk(const StepArgs& a, cudaStream_t stream) {
  const int splits = (a.dv + kRowsCta - 1) / kRowsCta;
  const long long ctas = (long long)a.N * a.H * splits;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.bf16)
    pool_step_kernel<DK, true><<<(unsigned)ctas, kStepThreads, 0, stream>>>(a, splits);
  else
    pool_step_kernel<DK, false><<<(unsigned)ctas, kStepThreads, 0, stream>>>(a, splits);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pool_step(const StepArgs& a, cudaStream_t stream) {
  if ((long long)a.N * a.T == 0) return cudaSuccess;
  switch (a.dk) {
    case 16: return launch_dk<16>(a, stream);
    case 32: return launch_dk<32>(a, stream);
    case 64: return launch_dk<64>(a, stream);
    case 128: return launch_dk<128>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gdn
