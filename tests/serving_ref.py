"""Plain 64-bit references of the serving operators, from their definitions, and the inputs
that the tests share.

Error bounds of the attention (derived, not fitted).  With u = 2^-22 (fp32 sums on the
tensor cores truncate, so twice the rounding unit of fp32 and a factor for the order of the
sum), X_i = max_j scale sum_d |q_id| |k_jd| and A_ic = sum_j p_ij |v_jc| (p the exact
probabilities):

* a score is a sum of d products: off by at most (d + 8) u X_i;
* e^x, the running maximum's factors and the sums over n keys: a relative (n + 32) u each,
  in the numerator and in the denominator;
* so |delta lse_i| <= (d + 8) u X_i + (n + 32) u + u |lse_i|, and
  |delta o_ic| <= 2 A_ic ((d + 8) u X_i + (n + 32) u);
* in bf16 the probabilities are rounded once more for the value product, 2^-8 A_ic, and
  the output is rounded to bf16, 2^-8 |o_ic| (and 2^-8 of what it is off by already): bf16
  has 8 significant bits, so a value of 1 and a bit moves by up to half of 2^-7.
"""
import math

import numpy as np
import torch

U = 2.0 ** -22


def plan(ctx, new, tables, ring, state, bs, T):
    """gdn_paged_plan, request by request."""
    tables, ring = tables.copy(), ring.copy()
    before, nb, M = tables.copy(), len(ring), tables.shape[1]
    head, count = int(state[0]) % nb, min(max(int(state[1]), 0), nb)
    N = len(ctx)
    cu, seq, ok = np.zeros(N + 1, np.int64), np.zeros(N, np.int64), np.zeros(N, np.int64)
    slots, pos = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    wanted = taken = back = 0
    for n in range(N):
        c, x = max(int(ctx[n]), 0), int(new[n])
        old = min(-(-c // bs), M)
        cu[n + 1] = cu[n] + max(x, 0)
        if x < 0:
            for i in range(old):
                if count + back < nb:
                    ring[(head + count + back) % nb] = before[n, i]
                    back += 1
            continue
        fits = c + x <= M * bs
        need = -(-(c + x) // bs) - old if fits else 0
        start, wanted = wanted, wanted + need
        ok[n] = fits and (need == 0 or wanted <= count)
        if ok[n]:
            for i in range(need):
                tables[n, old + i] = ring[(head + start + i) % nb]
            taken += need
            seq[n] = c + x
        for i in range(x):
            t = cu[n] + i
            if t < T:
                p = c + i
                pos[t] = p
                if ok[n]:
                    slots[t] = int(tables[n, p // bs]) * bs + p % bs
    return dict(cu_seqlens=cu, seq_lens=seq, slot_map=slots, positions=pos, granted=ok,
                ring_state=np.array([(head + taken) % nb, count - taken + back]), block_tables=tables,
                free_ring=ring)


def attention(q, k, v, past, scale, window):
    """One request in 64 bits: q [L, Hq, d] at positions past + i over k, v [S, Hkv, d].
    Returns o, lse and the bounds' A and X."""
    q, k, v = (x.double().cpu() for x in (q, k, v))
    L, Hq, d = q.shape
    S, Hkv = k.shape[:2]
    o, A = torch.zeros(L, Hq, d, dtype=torch.float64), torch.zeros(L, Hq, d, dtype=torch.float64)
    lse = torch.full((L, Hq), -math.inf, dtype=torch.float64)
    X = torch.zeros(L, Hq, dtype=torch.float64)
    for i in range(L):
        p = past + i
        lo, hi = max(0, p - window + 1) if window else 0, min(p + 1, S)
        if hi <= lo:
            continue
        for h in range(Hq):
            kk, vv = k[lo:hi, h * Hkv // Hq], v[lo:hi, h * Hkv // Hq]
            x = scale * (kk @ q[i, h])
            X[i, h] = scale * (kk.abs() @ q[i, h].abs()).max()
            lse[i, h] = torch.logsumexp(x, 0)
            w = torch.exp(x - lse[i, h])
            o[i, h] = w @ vv
            A[i, h] = w @ vv.abs()
    return o, lse, A, X


def bounds(o, lse, A, X, d, n, bf16):
    """Elementwise error bounds of out and lse."""
    s = (d + 8) * U * X + (n + 32) * U
    t = 2 * A * s[..., None]
    if bf16:
        t = t + 2.0 ** -8 * A
        t = t + 2.0 ** -8 * (o.abs() + t)
    return t, s + U * lse.abs()


def pages(lens, heads, d, block, dtype, seed, dev, junk=math.nan, spare=3, margin=1):
    """Caches whose unused places hold `junk`, the block tables (unused entries out of
    range), and each request's keys and values."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-x // block) for x in lens]
    nb, M = sum(held) + spare, max(held + [0]) + margin
    ids = torch.randperm(nb, generator=g).tolist()
    kc = torch.full((nb, block, heads, d), junk, dtype=dtype)
    vc = kc.clone()
    tables = torch.full((len(lens), M), -7, dtype=torch.int32)
    tables[:, -1] = 1 << 30
    keys, values, at = [], [], 0
    for n, x in enumerate(lens):
        k = torch.randn(x, heads, d, generator=g).to(dtype)
        v = torch.randn(x, heads, d, generator=g).to(dtype)
        for j in range(held[n]):
            b = ids[at + j]
            tables[n, j] = b
            part = slice(j * block, min(x, (j + 1) * block))
            kc[b, :part.stop - part.start] = k[part]
            vc[b, :part.stop - part.start] = v[part]
        at += held[n]
        keys.append(k)
        values.append(v)
    return kc.to(dev), vc.to(dev), tables.to(dev), keys, values
