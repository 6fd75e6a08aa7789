// The serving step's bookkeeping on the GPU: block tables, slot map and offsets from
// request lengths (gdn_paged_plan), and the write of new keys and values into the paged
// cache (gdn_paged_write).
#include <cuda_runtime.h>

#include "early_launch.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

// ------------------------------------------------------------------------- plan --
// With old_n = ceil(ctx_n / b) and need_n = ceil((ctx_n + new_n) / b) - old_n, three
// prefix sums over the requests (new tokens, needed blocks, released blocks) say where
// each request's tokens, its entries of the free ring and its released blocks lie; each
// token, new table entry and released block is then independent of the others.
//
// Bound by launch and memory latency: about 1 MB moves for 4096 requests and 65,000
// tokens.  So it is one launch with no communication between CTAs: every CTA scans all
// requests itself (two loads a request, 2048 requests a round) and takes a stripe of
// the tokens, table entries and released blocks, finding an item's request by binary
// search in the round's prefix sums in shared memory.  In-place updates cannot race: the
// entries that a call writes (table entries from old_n on, ring positions past the free
// range) are none of those it reads.
//
// Measured: 8 requests 4.5 us, 4096 requests with 65,000 new tokens 16 us.
constexpr int kPlanThreads = 512;
constexpr int kPlanPer = 4;                          // requests a thread holds
constexpr int kPlanChunk = kPlanThreads * kPlanPer;  // requests a round

struct Sum3 {
  long long tok;
  int need, back;
};
__device__ __forceinline__ Sum3 operator+(const Sum3& a, const Sum3& b) {
  return Sum3{a.tok + b.tok, a.need + b.need, a.back + b.back};
}
__device__ __forceinline__ Sum3 shfl_up(const Sum3& a, int o) {
  return Sum3{__shfl_up_sync(0xffffffffu, a.tok, o), __shfl_up_sync(0xffffffffu, a.need, o),
              __shfl_up_sync(0xffffffffu, a.back, o)};
}

// Last i in [0, n) with pre[i] <= x (pre non-decreasing, pre[0] <= x).
__device__ __forceinline__ int find(const int* pre, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int sat32(long long x) {
  return x > 0x7fffffffLL ? 0x7fffffff : (int)x;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PlanArgs a) {
  __shared__ int tok0[kPlanChunk + 1], need0[kPlanChunk + 1], back0[kPlanChunk + 1];
  __shared__ unsigned char ok[kPlanChunk];
  __shared__ Sum3 wsum[kPlanThreads / 32];
  __shared__ int taken_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_next_kernel_start();
  after_previous_kernel();
  const long long cap = (long long)a.max_blocks * a.block_size;
  const int bs = a.block_size, nb = a.num_blocks;
  int head = a.ring_in[0] % nb;
  if (head < 0) head += nb;
  const int count = min(max(a.ring_in[1], 0), nb);
  const int stride = gridDim.x * kPlanThreads;
  const int me = blockIdx.x * kPlanThreads + tid;
  if (tid == 0) taken_s = 0;
  Sum3 carry{0, 0, 0};

  for (int n0 = 0, round = 0; n0 < a.N; n0 += kPlanChunk, ++round) {
    const int nn = min(kPlanChunk, a.N - n0);
    const bool writer = round % gridDim.x == blockIdx.x;
    Sum3 mine[kPlanPer], sum{0, 0, 0};
    int ctx[kPlanPer], add[kPlanPer];
    bool fits[kPlanPer], done[kPlanPer];
#pragma unroll
    for (int u = 0; u < kPlanPer; ++u) {
      const int n = n0 + tid * kPlanPer + u;
      const bool in = n < a.N;
      ctx[u] = in ? max(__ldg(a.context_lens + n), 0) : 0;
      const int nw = in ? __ldg(a.new_lens + n) : 0;
      done[u] = nw < 0;
      add[u] = max(nw, 0);
    }
#pragma unroll
    for (int u = 0; u < kPlanPer; ++u) {
      const long long end = (long long)ctx[u] + add[u];
      fits[u] = end <= cap;
      const int old = (int)min((long long)a.max_blocks, ((long long)ctx[u] + bs - 1) / bs);
      mine[u].tok = add[u];
      mine[u].need = !done[u] && fits[u] ? (int)((end + bs - 1) / bs) - old : 0;
      mine[u].back = done[u] ? old : 0;
      sum = sum + mine[u];
    }
    Sum3 inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sum3 y = shfl_up(inc, o);
      if (lane >= o) inc = inc + y;
    }
    __syncthreads();  // the previous round's readers of the shared arrays are done
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    Sum3 base = carry, all = carry;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) base = base + wsum[w];
      all = all + wsum[w];
    }
    Sum3 at{base.tok + inc.tok - sum.tok, base.need + inc.need - sum.need,
            base.back + inc.back - sum.back};
    int last_taken = 0;
#pragma unroll
    for (int u = 0; u < kPlanPer; ++u) {
      const int i = tid * kPlanPer + u, n = n0 + i;
      const int cum = at.need + mine[u].need;
      const bool grant = !done[u] && fits[u] && (mine[u].need == 0 || cum <= count);
      if (grant && mine[u].need > 0) last_taken = cum;
      if (n < a.N) {
        tok0[i] = sat32(at.tok);
        need0[i] = at.need;
        back0[i] = at.back;
        ok[i] = grant;
        if (writer) {
          a.cu_seqlens[n] = sat32(at.tok);
          a.seq_lens[n] = grant ? (int)((long long)ctx[u] + add[u]) : 0;
          a.granted[n] = grant;
        }
      }
      at = at + mine[u];
    }
    if (tid == 0) {
      tok0[nn] = sat32(all.tok);
      need0[nn] = all.need;
      back0[nn] = all.back;
    }
    if (last_taken > 0) atomicMax(&taken_s, last_taken);
    __syncthreads();

    // tokens: a slot in the request's last held block, or in one of its new ones
    const int t_end = min(tok0[nn], a.T);
    for (int t = tok0[0] + me; t < t_end; t += stride) {
      const int i = find(tok0, nn, t), n = n0 + i;
      const long long pos = (long long)max(__ldg(a.context_lens + n), 0) + (t - tok0[i]);
      int slot = -1;
      if (ok[i]) {
        const int blk = (int)(pos / bs), old = (max(__ldg(a.context_lens + n), 0) + bs - 1) / bs;
        const int id = blk < old ? a.block_tables[(size_t)n * a.max_blocks + blk]
                                 : a.free_ring[((long long)head + need0[i] + (blk - old)) % nb];
        if (id >= 0 && id < nb) slot = (int)((long long)id * bs + (pos - (long long)blk * bs));
      }
      a.slot_map[t] = slot;
      a.positions[t] = sat32(pos);
      if (stride > 0x7fffffff - t) break;
    }
    // new table entries, from the front of the ring
    const int e_end = min(need0[nn], count);
    for (int e = need0[0] + me; e < e_end; e += stride) {
      const int i = find(need0, nn, e), n = n0 + i;
      if (ok[i]) {
        const int old = (max(__ldg(a.context_lens + n), 0) + bs - 1) / bs;
        a.block_tables[(size_t)n * a.max_blocks + old + (e - need0[i])] =
            a.free_ring[((long long)head + e) % nb];
      }
      if (stride > 0x7fffffff - e) break;
    }
    // released blocks, to the end of the ring (never past its capacity)
    const int r_end = min(back0[nn], nb - count);
    for (int r = back0[0] + me; r < r_end; r += stride) {
      const int i = find(back0, nn, r), n = n0 + i;
      a.free_ring[((long long)head + count + r) % nb] =
          a.block_tables[(size_t)n * a.max_blocks + (r - back0[i])];
      if (stride > 0x7fffffff - r) break;
    }
    carry = all;
  }
  // token rows past the last request
  for (long long t = min((long long)a.T, carry.tok) + me; t < a.T; t += stride) {
    a.slot_map[t] = -1;
    a.positions[t] = -1;
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    a.cu_seqlens[a.N] = sat32(carry.tok);
    a.ring_out[0] = (int)(((long long)head + taken_s) % nb);
    a.ring_out[1] = count - taken_s + min(carry.back, nb - count);
  }
}

// ------------------------------------------------------------------------ write --
// cache[slot_t] = row_t for keys and values: a copy, bound by HBM.  A thread moves
// kWriteVecs 16-byte pieces of both, all loads in flight before the first store.
// Measured: 32,768 tokens of 8 heads of 128 in bf16 40.8 us, 97 % of the copy rate.
constexpr int kWriteThreads = 256;
constexpr int kWriteVecs = 4;

__global__ void __launch_bounds__(kWriteThreads)
paged_write_kernel(const uint8_t* __restrict__ k, const uint8_t* __restrict__ v,
                   const int32_t* __restrict__ slot_map, uint8_t* __restrict__ kc,
                   uint8_t* __restrict__ vc, long long k_stride, long long v_stride,
                   unsigned row_vecs, long long total, long long slots) {
  let_next_kernel_start();
  after_previous_kernel();
  const long long base = (long long)blockIdx.x * (kWriteThreads * kWriteVecs) + threadIdx.x;
  uint4 kk[kWriteVecs], vv[kWriteVecs];
  long long to[kWriteVecs];
#pragma unroll
  for (int u = 0; u < kWriteVecs; ++u) {
    const long long idx = base + u * kWriteThreads;
    to[u] = -1;
    if (idx < total) {
      const long long t = idx / row_vecs;
      const unsigned c = (unsigned)(idx - t * row_vecs);
      const long long slot = __ldg(slot_map + t);
      if (slot >= 0 && slot < slots) {
        to[u] = (slot * row_vecs + c) * 16;
        kk[u] = *reinterpret_cast<const uint4*>(k + t * k_stride + (size_t)c * 16);
        vv[u] = *reinterpret_cast<const uint4*>(v + t * v_stride + (size_t)c * 16);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kWriteVecs; ++u)
    if (to[u] >= 0) {
      *reinterpret_cast<uint4*>(kc + to[u]) = kk[u];
      *reinterpret_cast<uint4*>(vc + to[u]) = vv[u];
    }
}

}  // namespace

int sm_count() {
  constexpr int kMaxDev = 64;
  static std::atomic<int> count[kMaxDev];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 152;
  if ((n = count[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
  count[dev].store(n, std::memory_order_relaxed);
  return n;
}

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t stream) {
  // one thread a token up to two CTAs an SM; requests are scanned by every CTA
  long long ctas = ((long long)(a.T > a.N ? a.T : a.N) + kPlanThreads - 1) / kPlanThreads;
  const int most = 2 * sm_count();
  if (ctas > most) ctas = most;
  if (ctas < 1) ctas = 1;
  return launch_early(paged_plan_kernel, dim3((unsigned)ctas), kPlanThreads, 0, stream, a);
}

cudaError_t launch_paged_write(const WriteArgs& a, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const unsigned row_vecs = (unsigned)(a.row_bytes / 16);
  const long long total = (long long)a.T * row_vecs;
  const long long ctas = (total + kWriteThreads * kWriteVecs - 1) / (kWriteThreads * kWriteVecs);
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_early(paged_write_kernel, dim3((unsigned)ctas), kWriteThreads, 0, stream, (const uint8_t*)a.k,
                      (const uint8_t*)a.v, a.slot_map, (uint8_t*)a.k_cache, (uint8_t*)a.v_cache, a.k_stride,
                      a.v_stride, row_vecs, total, a.slots);
}

}  // namespace gdn
