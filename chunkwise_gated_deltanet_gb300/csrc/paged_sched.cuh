// Work split shared by the paged-attention kernels.
//
// The queries of one request that read one key/value head form rows (token, head of the
// group), M of which make a unit; a unit reads the tiles of BN cached tokens that its rows
// see.  All tiles of all units, in the order (request, key/value head, row block, tile), are
// one line that the CTAs share evenly and contiguously, so that they end together whatever
// the requests' lengths are, without the host knowing them.  A unit whose tiles lie in one
// CTA's share is written by it; one that a share boundary cuts is left as partial results
// (unnormalised sums with their running maximum and sum), which the combine kernel joins in
// the order of the shares, so results do not depend on timing.  A share has at most two
// partial results: the unit that its start cuts (slot 0) and the one that its end cuts
// (slot 1).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kSchedMax = 1024;  // requests of one launch

struct SchedArgs {
  const int32_t* seq_lens;    // of this launch's first request
  const int32_t* cu_seqlens;
  const int32_t* block_tables;
  int nn, T, g, Hkv, window, max_blocks;
  long long max_kv;           // max_blocks * block_size
  int rows_lo, rows_hi;       // requests with rows in (rows_lo, rows_hi] only
  int min_tiles;              // tiles a CTA takes at least (while there are that many)
};

struct Req {
  int q0, ql, kl;
  int rows;  // query rows a key/value head, 0 if there is nothing to do
};

struct Item {
  int n, h, blk;  // request, key/value head, row block
  Req r;
  int tb, te;     // its tiles (of BN tokens) in this share; none if the rows see nothing
  bool whole;     // the share holds the whole unit
  int slot;       // partial-result slot otherwise
};

__device__ __forceinline__ Req load_req(const SchedArgs& s, int n) {
  Req r;
  const int a = min(max(__ldg(s.cu_seqlens + n), 0), s.T);
  const int b = min(max(__ldg(s.cu_seqlens + n + 1), a), s.T);
  r.q0 = a;
  r.ql = b - a;
  r.kl = (int)min((long long)max(__ldg(s.seq_lens + n), 0), s.max_kv);
  const long long rows = (long long)r.ql * s.g;
  r.rows = rows > s.rows_lo && rows <= s.rows_hi ? (int)rows : 0;
  return r;
}

template <int M, int BN>
struct Sched {
  SchedArgs s;
  const long long* pre;  // tiles before each request (nn + 1 entries, shared memory)
  long long total, first, pos, end, unit0;
  int G, cta, n, h, blk;
  Req r;
  bool started;

  // Tiles [lo, lo + count) of row block `b`; count >= 1 so that a block that sees nothing
  // is still written (`empty`).
  __device__ __forceinline__ int tiles(const Req& q, int b, int* lo, bool* empty) const {
    const int row0 = b * M, row1 = min(q.rows, row0 + M) - 1;
    const int p0 = q.kl - q.ql + row0 / s.g, hi = q.kl - q.ql + row1 / s.g + 1;
    const int l = s.window > 0 ? max(0, p0 - s.window + 1) : 0;
    *empty = hi <= 0;
    *lo = *empty ? 0 : l / BN;
    return *empty ? 1 : (hi + BN - 1) / BN - *lo;
  }
  __device__ __forceinline__ static int blocks(const Req& q) { return (q.rows + M - 1) / M; }

  // Whole CTA of NT threads: prefix sums of the requests' tiles into `pre_smem`.
  template <int NT>
  __device__ void init(const SchedArgs& args, long long* pre_smem, long long* warp_smem, int cta_id,
                       int grid) {
    s = args;
    pre = pre_smem;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long carry = 0;
    for (int n0 = 0; n0 < s.nn; n0 += NT) {
      long long x = 0;
      if (n0 + tid < s.nn) {
        const Req q = load_req(s, n0 + tid);
        const int nb = blocks(q);
        int lo;
        bool e;
        for (int b = 0; b < nb; ++b) x += tiles(q, b, &lo, &e);
        x *= s.Hkv;
      }
      long long inc = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (n0 > 0) __syncthreads();
      if (lane == 31) warp_smem[warp] = inc;
      __syncthreads();
      long long base = carry;
      for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) base += warp_smem[w];
        carry += warp_smem[w];
      }
      if (n0 + tid < s.nn) pre_smem[n0 + tid] = base + inc - x;
    }
    if (tid == 0) pre_smem[s.nn] = carry;
    __syncthreads();
    total = carry;
    const long long want = (total + s.min_tiles - 1) / s.min_tiles;
    G = (int)min((long long)grid, max(want, 1LL));
    cta = cta_id;
    first = cta < G ? share(cta) : total;
    pos = first;
    end = cta < G ? share(cta + 1) : total;
    started = false;
  }
  __device__ __forceinline__ long long share(int c) const { return total * c / G; }

  // Request, head, row block and start of the unit that holds tile `x`.
  __device__ void locate(long long x) {
    int lo = 0, hi = s.nn;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= x)
        lo = mid;
      else
        hi = mid;
    }
    n = lo;
    r = load_req(s, n);
    const long long per = (pre[n + 1] - pre[n]) / s.Hkv;
    long long rem = x - pre[n];
    h = (int)(rem / per);
    rem -= per * h;
    int l;
    bool e;
    for (blk = 0;; ++blk) {
      const int c = tiles(r, blk, &l, &e);
      if (rem < c) break;
      rem -= c;
    }
    unit0 = x - rem;
  }

  // Next piece of this CTA's share; the same for every thread that calls it.
  __device__ bool next(Item* it) {
    if (pos >= end) return false;
    if (!started) {
      locate(pos);
      started = true;
    } else {
      if (++blk == blocks(r)) {
        blk = 0;
        if (++h == s.Hkv) {
          h = 0;
          do {
            r = load_req(s, ++n);
          } while (r.rows == 0);
        }
      }
      unit0 = pos;
    }
    int lo;
    bool empty;
    const int c = tiles(r, blk, &lo, &empty);
    const long long stop = min(unit0 + c, end);
    it->n = n;
    it->h = h;
    it->blk = blk;
    it->r = r;
    it->tb = empty ? 0 : lo + (int)(pos - unit0);
    it->te = empty ? 0 : lo + (int)(stop - unit0);
    it->whole = pos == unit0 && stop == unit0 + c;
    it->slot = 2 * cta + (unit0 > first ? 1 : 0);
    pos = stop;
    return true;
  }
};

}  // namespace
}  // namespace gdn
