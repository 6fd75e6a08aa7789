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
//
// With WAVES, a launch whose caches do not fit L2 first gives out whole units in waves, unit
// w * CTAs + c to CTA c (odd waves the other way round), and shares only the last one to two
// waves as above.  The CTAs then work on neighbouring row blocks of a few heads at a time
// and read their keys and values from L2; contiguous shares would stream every head's cache
// from HBM at once.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {

struct SchedArgs {
  const int32_t* seq_lens;    // of this launch's first request
  const int32_t* cu_seqlens;
  const int32_t* block_tables;
  int nn, T, g, Hkv, window, max_blocks;
  long long max_kv;           // max_blocks * block_size
  int rows_lo, rows_hi;       // requests with rows in (rows_lo, rows_hi] only
  int min_tiles;              // tiles a CTA takes at least (while there are that many)
  long long wave_tokens;      // WAVES: cached tokens (all heads) above which waves are used
};

namespace {

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

// Shared memory of a scheduler.
template <int NMAX, bool WAVES>
struct SchedMem {
  long long pre[NMAX + 1];            // tiles before each request
  long long warp[32];
  int units[WAVES ? NMAX + 1 : 1];    // units before each request
  int warp_u[WAVES ? 32 : 1];
};

// M rows a unit, BN tokens a tile, NMAX requests a launch.
template <int M, int BN, int NMAX, bool WAVES>
struct Sched {
  using Mem = SchedMem<NMAX, WAVES>;
  static constexpr int kM = M;
  SchedArgs s;
  const Mem* mem;
  long long total, base, first, pos, end, unit0;
  int G, cta, n, h, blk;
  int waves, wave;
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

  // Whole CTA of NT threads: prefix sums of the requests' tiles and units into `m`.
  template <int NT>
  __device__ void init(const SchedArgs& args, Mem* m, int cta_id, int grid) {
    s = args;
    mem = m;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long carry = 0, tokens = 0;
    int carry_u = 0;
    for (int n0 = 0; n0 < s.nn; n0 += NT) {
      long long x = 0;
      int u = 0;
      if (n0 + tid < s.nn) {
        const Req q = load_req(s, n0 + tid);
        const int nb = blocks(q);
        int lo;
        bool e;
        for (int b = 0; b < nb; ++b) x += tiles(q, b, &lo, &e);
        x *= s.Hkv;
        u = nb * s.Hkv;
        if (WAVES && nb) tokens += q.kl;
      }
      long long inc = x;
      int inc_u = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
        if (WAVES) {
          const int yu = __shfl_up_sync(0xffffffffu, inc_u, o);
          if (lane >= o) inc_u += yu;
        }
      }
      if (n0 > 0) __syncthreads();
      if (lane == 31) {
        m->warp[warp] = inc;
        if (WAVES) m->warp_u[warp] = inc_u;
      }
      __syncthreads();
      long long before = carry;
      int before_u = carry_u;
      for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += m->warp[w];
        carry += m->warp[w];
        if (WAVES) {
          if (w < warp) before_u += m->warp_u[w];
          carry_u += m->warp_u[w];
        }
      }
      if (n0 + tid < s.nn) {
        m->pre[n0 + tid] = before + inc - x;
        if (WAVES) m->units[n0 + tid] = before_u + inc_u - u;
      }
    }
    if (tid == 0) {
      m->pre[s.nn] = carry;
      if (WAVES) m->units[s.nn] = carry_u;
    }
    __syncthreads();
    total = carry;
    const long long want = (total + s.min_tiles - 1) / s.min_tiles;
    G = (int)min((long long)grid, max(want, 1LL));
    cta = cta_id;
    base = 0;
    waves = 0;
    if (WAVES) {
      // cached tokens of the requests, over the CTA
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) tokens += __shfl_xor_sync(0xffffffffu, tokens, o);
      if (lane == 0) m->warp[warp] = tokens;
      __syncthreads();
      tokens = 0;
      for (int w = 0; w < NT / 32; ++w) tokens += m->warp[w];
      if (tokens > s.wave_tokens) waves = max(carry_u / G - 1, 0);
      if (waves > 0) {
        find_unit(waves * G);
        base = unit0;
      }
    }
    wave = 0;
    first = cta < G ? share(cta) : total;
    pos = first;
    end = cta < G ? share(cta + 1) : total;
    if (cta >= G) waves = 0;
    started = false;
  }
  __device__ __forceinline__ long long share(int c) const { return base + (total - base) * c / G; }

  // Request, head, row block and first tile of unit `u`.
  __device__ void find_unit(int u) {
    int lo = 0, hi = s.nn;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (mem->units[mid] <= u)
        lo = mid;
      else
        hi = mid;
    }
    n = lo;
    r = load_req(s, n);
    const int rem = u - mem->units[n], nb = blocks(r);
    h = rem / nb;
    blk = rem - h * nb;
    unit0 = mem->pre[n] + (mem->pre[n + 1] - mem->pre[n]) / s.Hkv * h;
    int l;
    bool e;
    for (int b = 0; b < blk; ++b) unit0 += tiles(r, b, &l, &e);
  }

  // Request, head, row block and start of the unit that holds tile `x`.
  __device__ void locate(long long x) {
    int lo = 0, hi = s.nn;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (mem->pre[mid] <= x)
        lo = mid;
      else
        hi = mid;
    }
    n = lo;
    r = load_req(s, n);
    const long long per = (mem->pre[n + 1] - mem->pre[n]) / s.Hkv;
    long long rem = x - mem->pre[n];
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
    if (WAVES && wave < waves) {
      find_unit(wave * G + (wave & 1 ? G - 1 - cta : cta));
      ++wave;
      int lo;
      bool empty;
      const int c = tiles(r, blk, &lo, &empty);
      it->n = n;
      it->h = h;
      it->blk = blk;
      it->r = r;
      it->tb = empty ? 0 : lo;
      it->te = empty ? 0 : lo + c;
      it->whole = true;
      it->slot = 0;
      return true;
    }
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
