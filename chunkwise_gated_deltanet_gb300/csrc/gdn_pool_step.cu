// The gated delta rule over a few new tokens per request, on a pool of states
// (gdn_recurrent_step): for request n with tokens cu[n] .. cu[n+1] and state
// S = pool[state_index[n]], for every token in order and every value head h
//
//     p = S k,  u = beta (v - alpha p),  S <- alpha S + u k^T,  o = S q
//
// (Nyysyyan, "Gated-DeltaNet" section, first equation block), with key head
// h / (H / Hk).  The state is read once and written once however many tokens there are.
//
// For a few tokens this is bound by HBM (8 dk dv bytes a (request, head)); the arithmetic on
// the CUDA cores passes it at about a dozen tokens, so it is kept short:
//
// * S is held as A S~ with A the product of the alphas since the tokens were staged, which
//   leaves one multiply-add an element for the update:
//       u = beta (v - A p~),  S~ <- S~ + (u / A) k^T,  o = A s~ + u (k . q),
//   p~ = S~ k, s~ = S~ q.  The last A is multiplied in at the end of a stage.  Where A would
//   fall below 2^-60 within a stage (strong decay, alpha = 0), S is scaled token by token.
// * Every product is a packed pair (fma.rn.f32x2).
// * A lane holds 4 rows of S, an eighth of the columns each, so that a read of k or q from
//   shared memory serves 4 rows; the 8 sums of a row quartet are reduced over the 8 lanes
//   together (7 shuffles, each lane ends with one of them).
//
// A CTA has one (request, head): a warp for every 16 rows.  k, q, v are staged as fp32 in
// shared memory, kStage tokens at a time, and outputs leave through it in whole lines.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kStage = 16;  // tokens staged at a time
constexpr int kRows = 4;    // rows a lane

template <bool BF16>
__device__ __forceinline__ float4 ld4f(const void* p, size_t i) {
  if (BF16) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(p) + i));
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  }
  return __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i));
}
template <bool BF16>
__device__ __forceinline__ void st4f(void* p, size_t i, float4 x) {
  if (BF16) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p) + i) =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) = x;
  }
}

__device__ __forceinline__ uint64_t both(float a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ float sum_of(uint64_t x) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
  return a + b;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <int DK>
struct StepSmem {
  float k[kStage][DK], q[kStage][DK];
  float alpha[kStage], beta[kStage], A[kStage], inv[kStage], kq[kStage];
  int slow;
};

// v and the outputs follow in dynamic shared memory: [kStage][dv] each.
template <int DK, bool BF16>
__global__ void __launch_bounds__(256, 2) pool_step_kernel(const __grid_constant__ StepArgs a) {
  constexpr int L = DK >= 32 ? 8 : 4;  // lanes a row
  constexpr int NP = DK / L / 2;       // pairs of S a lane and row
  __shared__ __align__(16) StepSmem<DK> sm;
  extern __shared__ __align__(16) float vo[];

  const int n = blockIdx.x / a.H, h = blockIdx.x - n * a.H, hk = h / (a.H / a.Hk);
  const int t0 = min(max(__ldg(a.cu_seqlens + n), 0), a.T);
  const int t1 = min(max(__ldg(a.cu_seqlens + n + 1), t0), a.T);
  if (t0 == t1) return;  // no tokens: the state stays as it is
  const int slot = __ldg(a.state_index + n);
  const int tid = threadIdx.x, nthreads = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int dv = a.dv, dv4 = dv / 4;
  if (slot < 0 || slot >= a.slots) {  // no state: the outputs are zeros
    for (int e = tid; e < (t1 - t0) * dv4; e += nthreads)
      st4f<BF16>(a.out, ((size_t)(t0 + e / dv4) * a.H + h) * dv + (e % dv4) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }
  float* vs = vo;
  float* os = vo + kStage * dv;
  // lane `sub` of a row group: columns 4 (sub + L i) .. + 3; rows row .. row + 3
  const int sub = lane % L;
  const int row = (warp * (32 / L) + lane / L) * kRows;
  const bool live = row < dv;
  const bool fresh = a.context_lens != nullptr && __ldg(a.context_lens + n) <= 0;
  float* S = a.pool + (((size_t)slot * a.H + h) * dv + row) * DK + 4 * sub;
  uint64_t s[kRows][NP];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int i = 0; i < NP; i += 2) {
      ulonglong2 x = make_ulonglong2(0, 0);
      if (live && !fresh) x = *reinterpret_cast<const ulonglong2*>(S + (size_t)r * DK + 2 * L * i);
      s[r][i] = x.x;
      s[r][i + 1] = x.y;
    }

  for (int tb = t0; tb < t1; tb += kStage) {
    const int nt = min(kStage, t1 - tb);
    for (int e = tid; e < nt * (DK / 4); e += nthreads) {
      const int j = e / (DK / 4), c = (e % (DK / 4)) * 4;
      *reinterpret_cast<float4*>(&sm.k[j][c]) = ld4f<BF16>(a.k, (size_t)(tb + j) * a.k_stride + hk * DK + c);
      *reinterpret_cast<float4*>(&sm.q[j][c]) = ld4f<BF16>(a.q, (size_t)(tb + j) * a.q_stride + hk * DK + c);
    }
    for (int e = tid; e < nt * dv4; e += nthreads) {
      const int j = e / dv4, c = (e - j * dv4) * 4;
      *reinterpret_cast<float4*>(vs + j * dv + c) =
          ld4f<BF16>(a.v, (size_t)(tb + j) * a.v_stride + (size_t)h * dv + c);
    }
    if (warp == 0) {
      float al = 1.f, be = 0.f;
      if (lane < nt) {
        al = expf(__ldg(a.log_alpha + (size_t)(tb + lane) * a.H + h));
        be = __ldg(a.beta + (size_t)(tb + lane) * a.H + h);
      }
      float A = al;
#pragma unroll
      for (int o = 1; o < kStage; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, A, o);
        if (lane >= o) A *= y;
      }
      const bool slow = __any_sync(0xffffffffu, !(A >= 0x1p-60f));
      if (slow) A = 1.f;
      if (lane < nt) {
        sm.alpha[lane] = al;
        sm.beta[lane] = be;
        sm.A[lane] = A;
        sm.inv[lane] = 1.f / A;
      }
      if (lane == 0) sm.slow = slow;
    }
    __syncthreads();
    // k . q of each staged token, a warp a token
    for (int j = warp; j < nt; j += nthreads >> 5) {
      float x = 0.f;
      for (int c = lane; c < DK; c += 32) x = fmaf(sm.k[j][c], sm.q[j][c], x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == 0) sm.kq[j] = x;
    }
    __syncthreads();
    const bool slow = sm.slow != 0;
    for (int j = 0; j < nt; ++j) {
      const float A = sm.A[j];
      if (slow) {
        const uint64_t al = both(sm.alpha[j]);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int i = 0; i < NP; ++i) s[r][i] = mul2(s[r][i], al);
      }
      uint64_t kk[NP];
      float x[2 * kRows];  // p~ of the rows, then s~
      {
        uint64_t p[kRows], q[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) p[r] = q[r] = 0;
#pragma unroll
        for (int i = 0; i < NP; i += 2) {
          const ulonglong2 k2 = *reinterpret_cast<const ulonglong2*>(&sm.k[j][4 * sub + 2 * L * i]);
          const ulonglong2 q2 = *reinterpret_cast<const ulonglong2*>(&sm.q[j][4 * sub + 2 * L * i]);
          kk[i] = k2.x;
          kk[i + 1] = k2.y;
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            p[r] = fma2(s[r][i], k2.x, p[r]);
            q[r] = fma2(s[r][i], q2.x, q[r]);
            p[r] = fma2(s[r][i + 1], k2.y, p[r]);
            q[r] = fma2(s[r][i + 1], q2.y, q[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          x[r] = sum_of(p[r]);
          x[kRows + r] = sum_of(q[r]);
        }
      }
      const float beta = sm.beta[j], inv = sm.inv[j], kq = sm.kq[j];
      float w[kRows];  // u / A of the four rows
      if (L == 8) {
        // lane `sub` ends with the total of x[sub]: halves exchanged with lanes 4, 2, 1 apart
        float y4[4], y2[2], y;
        const bool b4 = sub & 4, b2 = sub & 2, b1 = sub & 1;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          y4[i] = (b4 ? x[4 + i] : x[i]) + __shfl_xor_sync(0xffffffffu, b4 ? x[i] : x[4 + i], 4);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          y2[i] = (b2 ? y4[2 + i] : y4[i]) + __shfl_xor_sync(0xffffffffu, b2 ? y4[i] : y4[2 + i], 2);
        y = (b1 ? y2[1] : y2[0]) + __shfl_xor_sync(0xffffffffu, b1 ? y2[0] : y2[1], 1);
        // lanes 0-3: u of row `sub`; lanes 4-7: the output of row `sub` - 4
        const float vr = live ? vs[j * dv + row + (sub & 3)] : 0.f;
        const float u = beta * fmaf(-A, y, vr);
        const float ur = __shfl_sync(0xffffffffu, u, (lane & ~7) + (sub & 3));
        if (live && sub >= 4) os[j * dv + row + sub - 4] = fmaf(A, y, ur * kq);
        const float wr = ur * inv;
#pragma unroll
        for (int r = 0; r < kRows; ++r) w[r] = __shfl_sync(0xffffffffu, wr, (lane & ~7) + r);
      } else {
#pragma unroll
        for (int i = 0; i < 2 * kRows; ++i)
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float vr = live ? vs[j * dv + row + r] : 0.f;
          const float u = beta * fmaf(-A, x[r], vr);
          if (live && sub == 0) os[j * dv + row + r] = fmaf(A, x[kRows + r], u * kq);
          w[r] = u * inv;
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const uint64_t w2 = both(w[r]);
#pragma unroll
        for (int i = 0; i < NP; ++i) s[r][i] = fma2(w2, kk[i], s[r][i]);
      }
    }
    if (!slow) {
      const uint64_t A = both(sm.A[nt - 1]);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int i = 0; i < NP; ++i) s[r][i] = mul2(s[r][i], A);
    }
    __syncthreads();
    for (int e = tid; e < nt * dv4; e += nthreads) {
      const int j = e / dv4, c = (e - j * dv4) * 4;
      st4f<BF16>(a.out, ((size_t)(tb + j) * a.H + h) * dv + c, *reinterpret_cast<const float4*>(os + j * dv + c));
    }
  }
  if (live) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int i = 0; i < NP; i += 2)
        *reinterpret_cast<ulonglong2*>(S + (size_t)r * DK + 2 * L * i) = make_ulonglong2(s[r][i], s[r][i + 1]);
  }
}

template <int DK>
cudaError_t launch_dk(const StepArgs& a, cudaStream_t stream) {
  const long long ctas = (long long)a.N * a.H;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  constexpr int rows_warp = 32 / (DK >= 32 ? 8 : 4) * kRows;
  const int threads = 32 * ((a.dv + rows_warp - 1) / rows_warp);
  const int bytes = 2 * kStage * a.dv * 4;
  if (a.bf16)
    pool_step_kernel<DK, true><<<(unsigned)ctas, threads, bytes, stream>>>(a);
  else
    pool_step_kernel<DK, false><<<(unsigned)ctas, threads, bytes, stream>>>(a);
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
