// The gated delta rule over a few new tokens per request, on a pool of states
// (gdn_recurrent_step): for request n with tokens cu[n] .. cu[n+1] and state
// S = pool[state_index[n]], for every token in order and every value head h
//
//     p = S k,  u = beta (v - alpha p),  S <- alpha S + u k^T,  o = S q
//
// (Nyysyyan, "Gated-DeltaNet" section, first equation block), with key head
// h / (H / Hk).  The state is read once and written once however many tokens there are.
//
// For a few tokens this is bound by HBM (8 dk dv bytes a (request, head)).  Token by token on
// the CUDA cores the arithmetic passes that at a few tokens: 96 packed multiply-adds and as
// much again for reductions and operands, a warp, 16 rows and token (1 to 8 tokens x 256
// requests of 16 heads took 122 us, up to 64 tokens x 48 requests of 32 heads 183 us).  So
// tokens go kC = 8 at a time, in the chunk form with S0 the state before them, D_ts the product
// of alpha_{s+1} .. alpha_t and gamma_t that of alpha_0 .. alpha_t:
//
//     u_t = beta_t (v_t - gamma_t S0 k_t) - sum_{s<t} beta_t D_ts (k_t . k_s) u_s
//     o_t = gamma_t S0 q_t + sum_{s<=t} D_ts (q_t . k_s) u_s
//     S   = gamma_7 S0 + sum_s D_7s u_s k_s^T
//
// The products with S0 and the update run on mma.sync (m16n8k8, TF32) in three passes of
// two-part operands (hi hi + hi lo + lo hi, about 2^-22 relative, fp32 sums); the sums over
// s < t are eight steps in registers.  A warp has 16 rows of S in the accumulators' layout for
// the whole call.  The same registers are the products' left operand: an accumulator's columns
// 2 t and 2 t + 1 stand for the operand's t and t + 4, and the right operands are laid out in
// shared memory in that order, a 16-byte piece a lane (hi and lo of both values).  The next
// tokens' k, q, v come by cp.async under this chunk's products.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kC = 8;  // tokens at a time

template <bool BF16>
__device__ __forceinline__ void st1f(void* p, size_t i, float x) {
  if (BF16)
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else
    reinterpret_cast<float*>(p)[i] = x;
}

// x = hi + lo with hi of TF32's 11 significant bits; lo is cut to them by the product.
__device__ __forceinline__ uint32_t tf_hi(float x) { return __float_as_uint(x) & 0xffffe000u; }
__device__ __forceinline__ uint32_t tf_lo(float x, uint32_t hi) {
  return __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}
__device__ __forceinline__ uint4 tf_pair(float a, float b) {  // hi, hi, lo, lo
  const uint32_t ha = tf_hi(a), hb = tf_hi(b);
  return make_uint4(ha, hb, tf_lo(a, ha), tf_lo(b, hb));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c += a b in three passes; b as tf_pair has it.
__device__ __forceinline__ void mma_3(float (&c)[4], const uint32_t (&hi)[4], const uint32_t (&lo)[4], uint4 b) {
  mma_tf32(c, lo, b.x, b.y);
  mma_tf32(c, hi, b.z, b.w);
  mma_tf32(c, hi, b.x, b.y);
}

// 16 or 4 bytes into shared memory, zeros where there are none.
__device__ __forceinline__ void copy16(void* to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
               "l"(from), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(void* to, const void* from, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
               "l"(from), "r"(there ? 4 : 0)
               : "memory");
}

template <int DK, bool BF16>
struct StepSmem {
  static constexpr int kSize = BF16 ? 2 : 4, kPad = 16 / kSize;  // rows padded: other banks
  using El = typename std::conditional<BF16, __nv_bfloat16, float>::type;
  // the coming chunk's tokens as they are, zeros past the request's
  alignas(16) El k[kC][DK + kPad];
  alignas(16) El q[kC][DK + kPad];
  alignas(16) El v[kC][128 + kPad];
  alignas(16) float raw_la[kC];
  alignas(16) float raw_beta[kC];
  // right operands, a piece a lane (g = lane / 4, t = lane % 4) and 8 columns: k and q of token
  // g at the columns of the lane's accumulators, and k of tokens 2 t, 2 t + 1 at column g's
  alignas(16) uint4 kd[DK / 8][32], qd[DK / 8][32], ku[DK / 8][32];
  // of tokens 2 t, 2 t + 1 and s: beta_t D_ts k_t . k_s (s < t, else 0) of both, D_ts q_t . k_s
  // (s <= t) of both
  alignas(16) float4 m[kC][4];
  float decay[kC][kC];       // D_ts
  float part[8][16][kC + 1]; // a warp's part of k_i . k_j (rows 0-7) and q_i . k_j (8-15)
  float beta[kC], gamma[kC], last[kC];
};
// Column of an accumulator's entry: tile n of 8, column j of the tile.  A lane's entries of
// tiles 2 m and 2 m + 1 are the four consecutive columns 16 m + 4 t ..
__device__ __forceinline__ int col_of(int n, int j) {
  return 16 * (n >> 1) + 4 * (j >> 1) + 2 * (n & 1) + (j & 1);
}

template <int DK, bool BF16>
__global__ void __launch_bounds__(256, 2) pool_step_kernel(const __grid_constant__ StepArgs a) {
  constexpr int NT = DK / 8;  // column tiles of S
  __shared__ StepSmem<DK, BF16> sm;

  const int n = blockIdx.x / a.H, h = blockIdx.x - n * a.H, hk = h / (a.H / a.Hk);
  const int t0 = min(max(__ldg(a.cu_seqlens + n), 0), a.T);
  const int t1 = min(max(__ldg(a.cu_seqlens + n + 1), t0), a.T);
  if (t0 == t1) return;  // no tokens: the state stays as it is
  const int slot = __ldg(a.state_index + n);
  const int tid = threadIdx.x, nthreads = blockDim.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int warp = tid >> 5, nwarps = nthreads >> 5;
  const int dv = a.dv, row = warp * 16 + g;  // this lane's rows: row and row + 8
  if (slot < 0 || slot >= a.slots) {               // no state: the outputs are zeros
    for (int e = tid; e < (t1 - t0) * dv; e += nthreads)
      st1f<BF16>(a.out, ((size_t)(t0 + e / dv) * a.H + h) * dv + e % dv, 0.f);
    return;
  }
  const bool fresh = a.context_lens != nullptr && __ldg(a.context_lens + n) <= 0;
  using Sm = StepSmem<DK, BF16>;
  using El = typename Sm::El;
  auto stage = [&](int tb) {  // the chunk from token tb on
    constexpr int V = 16 / Sm::kSize;
    const El* k = reinterpret_cast<const El*>(a.k) + hk * DK;
    const El* q = reinterpret_cast<const El*>(a.q) + hk * DK;
    const El* v = reinterpret_cast<const El*>(a.v) + (size_t)h * dv;
    for (int e = tid; e < kC * (DK / V); e += nthreads) {
      const int j = e / (DK / V), c = (e % (DK / V)) * V;
      const bool in = tb + j < t1;
      const size_t at = in ? tb + j : tb;
      copy16(&sm.k[j][c], k + at * a.k_stride + c, in);
      copy16(&sm.q[j][c], q + at * a.q_stride + c, in);
    }
    for (int e = tid; e < kC * (dv / V); e += nthreads) {
      const int j = e / (dv / V), c = (e % (dv / V)) * V;
      const bool in = tb + j < t1;
      copy16(&sm.v[j][c], v + (size_t)(in ? tb + j : tb) * a.v_stride + c, in);
    }
    if (tid < 2 * kC) {
      const int j = tid & 7;
      const bool in = tb + j < t1;
      const size_t at = (size_t)(in ? tb + j : tb) * a.H + h;
      if (tid < kC)
        copy4(&sm.raw_la[j], a.log_alpha + at, in);
      else
        copy4(&sm.raw_beta[j], a.beta + at, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  stage(t0);
  float* S = a.pool + (((size_t)slot * a.H + h) * dv + row) * DK + 4 * t;
  float s[NT][4];
#pragma unroll
  for (int m = 0; m < NT; m += 2)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!fresh) x = *reinterpret_cast<const float4*>(S + (size_t)(8 * r) * DK + 8 * m);
      s[m][2 * r] = x.x;
      s[m][2 * r + 1] = x.y;
      s[m + 1][2 * r] = x.z;
      s[m + 1][2 * r + 1] = x.w;
    }

  for (int tb = t0; tb < t1; tb += kC) {
    const int nt = min(kC, t1 - tb);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    // from the staged tokens: the operands, the gates, and v of this lane's rows
    auto f = [](El x) { return (float)x; };
    for (int e = tid; e < NT * 32; e += nthreads) {
      const int m = e >> 5, lg = (e & 31) >> 2, lt = e & 3, c = col_of(m, 2 * lt), cg = col_of(m, lg);
      sm.kd[m][e & 31] = tf_pair(f(sm.k[lg][c]), f(sm.k[lg][c + 1]));
      sm.qd[m][e & 31] = tf_pair(f(sm.q[lg][c]), f(sm.q[lg][c + 1]));
      sm.ku[m][e & 31] = tf_pair(f(sm.k[2 * lt][cg]), f(sm.k[2 * lt + 1][cg]));
    }
    for (int e = tid; e < kC * kC; e += nthreads) {
      const int i = e >> 3, j = e & 7;  // D_ij, and in the row's end gamma_j and D_7j
      float x = 0.f;
      for (int u = j + 1; u <= i; ++u) x += sm.raw_la[u];
      sm.decay[i][j] = j > i ? 0.f : expf(x);
      if (i == kC - 1) {
        sm.last[j] = expf(x);
        float y = 0.f;
        for (int u = 0; u <= j; ++u) y += sm.raw_la[u];
        sm.gamma[j] = expf(y);
        sm.beta[j] = sm.raw_beta[j];
      }
    }
    float v[2][2];  // tokens 2 t, 2 t + 1 (second index)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int b = 0; b < 2; ++b) v[r][b] = f(sm.v[2 * t + b][row + 8 * r]);
    __syncthreads();
    if (tb + kC < t1) stage(tb + kC);
    // the tokens' products with each other: a warp takes every (warps)-th tile of columns
    {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
      for (int m = warp; m < NT; m += nwarps) {
        const uint4 kk = sm.kd[m][lane], qq = sm.qd[m][lane];
        const uint32_t hi[4] = {kk.x, qq.x, kk.y, qq.y}, lo[4] = {kk.z, qq.z, kk.w, qq.w};
        mma_3(c, hi, lo, kk);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sm.part[warp][g + 8 * (e >> 1)][2 * t + (e & 1)] = c[e];
    }
    __syncthreads();
    for (int e = tid; e < 2 * kC * kC; e += nthreads) {
      const int i = e >> 3, j = e & 7;  // row i of part, token j
      const int ti = i & 7;
      float dot = 0.f;
      for (int w = 0; w < min(nwarps, NT); ++w) dot += sm.part[w][i][j];
      float* to = reinterpret_cast<float*>(&sm.m[j][ti >> 1]) + (ti & 1);
      const float x = j > ti ? 0.f : sm.decay[ti][j] * dot;
      if (i >= kC)
        to[2] = x;
      else
        to[0] = j < ti ? sm.beta[ti] * x : 0.f;
    }

    float p[2][4], o[2][4];  // S0 k and S0 q of the 16 rows and 8 tokens, in two chains each
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) p[c][e] = o[c][e] = 0.f;
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      const float x[4] = {s[m][0], s[m][2], s[m][1], s[m][3]};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        hi[e] = tf_hi(x[e]);
        lo[e] = tf_lo(x[e], hi[e]);
      }
      mma_3(p[m & 1], hi, lo, sm.kd[m][lane]);
      mma_3(o[m & 1], hi, lo, sm.qd[m][lane]);
    }
    __syncthreads();  // m is there
    float u[2][2], y[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float beta = sm.beta[2 * t + b], gamma = sm.gamma[2 * t + b];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        u[r][b] = beta * fmaf(-gamma, p[0][2 * r + b] + p[1][2 * r + b], v[r][b]);
        y[r][b] = gamma * (o[0][2 * r + b] + o[1][2 * r + b]);
      }
    }
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const float4 m = sm.m[j][t];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float x = __shfl_sync(0xffffffffu, u[r][j & 1], (lane & ~3) + (j >> 1));
        // by selection: a later token's value, whatever it is, adds nothing to an earlier one
        if (2 * t > j) u[r][0] = fmaf(-m.x, x, u[r][0]);
        if (2 * t + 1 > j) u[r][1] = fmaf(-m.y, x, u[r][1]);
        if (2 * t >= j) y[r][0] = fmaf(m.z, x, y[r][0]);
        if (2 * t + 1 >= j) y[r][1] = fmaf(m.w, x, y[r][1]);
      }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
      if (2 * t + b < nt) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
          st1f<BF16>(a.out, ((size_t)(tb + 2 * t + b) * a.H + h) * dv + row + 8 * r, y[r][b]);
      }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float w = sm.last[2 * t + b];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float x = w * u[r][b];
        hi[2 * b + r] = tf_hi(x);
        lo[2 * b + r] = tf_lo(x, hi[2 * b + r]);
      }
    }
    const float gamma = sm.gamma[kC - 1];
#pragma unroll
    for (int m = 0; m < NT; ++m) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[m][e] *= gamma;
      mma_3(s[m], hi, lo, sm.ku[m][lane]);
    }
  }
#pragma unroll
  for (int m = 0; m < NT; m += 2)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      *reinterpret_cast<float4*>(S + (size_t)(8 * r) * DK + 8 * m) =
          make_float4(s[m][2 * r], s[m][2 * r + 1], s[m + 1][2 * r], s[m + 1][2 * r + 1]);
}

template <int DK>
cudaError_t launch_dk(const StepArgs& a, cudaStream_t stream) {
  const long long ctas = (long long)a.N * a.H;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int threads = 32 * (a.dv / 16);
  if (a.bf16)
    pool_step_kernel<DK, true><<<(unsigned)ctas, threads, 0, stream>>>(a);
  else
    pool_step_kernel<DK, false><<<(unsigned)ctas, threads, 0, stream>>>(a);
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
