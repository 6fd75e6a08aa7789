"""The serving operators of a hybrid stack (gated-delta layers beside attention layers) and
their plain forms.

  plan    block tables, slot map and offsets of one step, built on the GPU from request lengths
  write   the step's new keys and values into the paged cache
  attend  attention of each request's new tokens over its paged cache (causal, optional window)
  step    the gated delta rule over a few new tokens per request, on a pool of states

``run`` computes a case in plain torch operations (fp32), or with ``own`` through this
repository's package; ``exact`` computes it in 64 bits from the definition.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases --
def listed():
    return [
        # a small server between two tokens: 8 requests, one new token each; pure latency
        dict(name="plan_n8_decode", op="plan", n=8, ctx_hi=2048, new_hi=1, block=16, done=0.0, spare=2.0,
             lens_seed=1),
        # a full scheduler step: thousands of requests, prefill chunks among single tokens, some
        # requests finished, and too few free blocks for the last ones
        dict(name="plan_n4096_mixed", op="plan", n=4096, ctx_hi=8192, new_hi=64, block=16, done=0.05,
             spare=0.97, lens_seed=2),
        # the cache write of a small decode batch
        dict(name="write_t37_bf16", op="write", tokens=37, kv_heads=4, d=128, dtype="bf16", block=16,
             fused=True, drop=0.0),
        # the cache write of a long prefill (the 32768-token workload), keys and values read as
        # slices of one fused projection
        dict(name="write_t32768_bf16", op="write", tokens=32768, kv_heads=8, d=128, dtype="bf16", block=64,
             fused=True, drop=0.02),
        # one token for three short requests: latency
        dict(name="attend_n3_decode", op="attend", n=3, q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=700, heads=16,
             kv_heads=4, d=128, dtype="bf16", block=16, window=0, lens_seed=3),
        # one token for each of 256 requests of 64 to 2048 tokens: the packed workload, decoding
        dict(name="attend_n256_decode", op="attend", n=256, q_lo=1, q_hi=1, ctx_lo=64, ctx_hi=2048, heads=16,
             kv_heads=4, d=128, dtype="bf16", block=16, window=0, lens_seed=4),
        # one request far into a long document, four tokens at once: few rows, a long axis
        dict(name="attend_n1_q4_long", op="attend", n=1, q_lo=4, q_hi=4, ctx_lo=131071, ctx_hi=131071,
             heads=32, kv_heads=4, d=128, dtype="bf16", block=64, window=0, lens_seed=5),
        # chunked prefill: some 2000 new tokens of two requests over tens of thousands of cached ones
        dict(name="attend_n2_chunk2048", op="attend", n=2, q_lo=1900, q_hi=2048, ctx_lo=20000,
             ctx_hi=30720, heads=32, kv_heads=8, d=128, dtype="bf16", block=16, window=0, lens_seed=6),
        # the fp32 sizes (2 sequences, 4 heads of 64), a chunk with a sliding window
        dict(name="attend_f32_window", op="attend", n=2, q_lo=200, q_hi=320, ctx_lo=500, ctx_hi=1024, heads=4,
             kv_heads=2, d=64, dtype="f32", block=8, window=256, lens_seed=7),
        # a few requests of an fp32 model, one token each
        dict(name="step_n4_f32", op="step", n=4, t_lo=1, t_hi=1, k_heads=4, heads=4, dk=64, dv=64, dtype="f32",
             fresh=0.0, lens_seed=8),
        # a decode batch with drafted tokens: 256 requests, 1 to 8 tokens each, shared key heads
        dict(name="step_n256_draft", op="step", n=256, t_lo=1, t_hi=8, k_heads=8, heads=16, dk=128, dv=128,
             dtype="bf16", fresh=0.0, lens_seed=9),
        # a mixed step: short prompt chunks, some of them of new requests
        dict(name="step_n48_chunk64", op="step", n=48, t_lo=1, t_hi=64, k_heads=16, heads=32, dk=128, dv=128,
             dtype="bf16", fresh=0.25, lens_seed=10),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("plan", "write", "attend", "attend", "attend", "step", "step"))
    seed = rng.randrange(1 << 30)
    if op == "plan":
        return dict(op=op, n=_log_int(rng, 1, 4096), ctx_hi=_log_int(rng, 1, 8192), new_hi=_log_int(rng, 1, 64),
                    block=rng.choice((8, 16, 24, 64, 128)), done=rng.choice((0.0, 0.1, 0.4)),
                    spare=rng.choice((0.6, 1.0, 3.0)), lens_seed=seed)
    if op == "write":
        return dict(op=op, tokens=_log_int(rng, 1, 32768), kv_heads=rng.choice((1, 2, 3, 4, 8)),
                    d=rng.choice((16, 32, 64, 128)), dtype=rng.choice(("bf16", "f32")),
                    block=rng.choice((8, 16, 48, 128)), fused=rng.random() < 0.5, drop=rng.choice((0.0, 0.1)))
    if op == "attend":
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        d = rng.choice((64, 128, 128, 128, 16, 32))
        kv_heads = rng.choice((1, 2, 4, 8))
        heads = kv_heads * rng.choice((1, 2, 3, 4, 8))
        q_hi = _log_int(rng, 1, 2048)
        ctx_hi = _log_int(rng, 1, 32768)
        n = _log_int(rng, 1, 256)
        top = 2e9 if dtype == "bf16" else 2e8  # query-key pairs of all heads, padded: at most half the largest case's
        n = max(1, min(n, int(top / (heads * q_hi * (ctx_hi + q_hi))), int(1e9 / ((ctx_hi + q_hi) * kv_heads * d))))
        q_hi = max(1, min(q_hi, int(top / (n * heads * (ctx_hi + q_hi)))))
        return dict(op=op, n=n, q_lo=rng.choice((1, max(1, q_hi // 2), q_hi)), q_hi=q_hi,
                    ctx_lo=rng.choice((0, ctx_hi // 2)), ctx_hi=ctx_hi, heads=heads, kv_heads=kv_heads, d=d,
                    dtype=dtype, block=rng.choice((8, 16, 24, 32, 64, 128, 256)),
                    window=rng.choice((0, 0, 0, _log_int(rng, 1, 4096))), lens_seed=seed)
    d = rng.choice((16, 32, 64, 128, 128))
    t_hi = _log_int(rng, 1, 64)
    heads = rng.choice((4, 8, 16, 32))
    n = _log_int(rng, 1, 256)
    n = max(1, min(n, int(256 * 16 * 8 * 1.1 / (heads * max(t_hi, 8)))))
    return dict(op="step", n=n, t_lo=rng.choice((1, t_hi)), t_hi=t_hi, k_heads=heads // rng.choice((1, 2, 4)),
                heads=heads, dk=d, dv=rng.choice((d, d, 16, 64, 128)), dtype=rng.choice(("bf16", "f32")),
                fresh=rng.choice((0.0, 0.5)), lens_seed=seed)


def _lengths(case, lo, hi, salt):
    r = random.Random(case["lens_seed"] * 4 + salt)
    return [r.randint(lo, hi) for _ in range(case["n"])]


def _plan_lengths(case):
    r = random.Random(case["lens_seed"])
    ctx, new = [], []
    for _ in range(case["n"]):
        done = r.random() < case["done"]
        ctx.append(r.randint(1 if done else 0, case["ctx_hi"]))
        new.append(-1 if done else 1 if r.random() < 0.5 else r.randint(1, case["new_hi"]))
    return ctx, new


def _ceil(a, b):
    return -(-a // b)


# ----------------------------------------------------------------- the inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


def prepare(case, seed):
    return {"plan": _prepare_plan, "write": _prepare_write, "attend": _prepare_attend,
            "step": _prepare_step}[case["op"]](case, seed)


def _prepare_plan(case, seed):
    g = _gen(seed)
    ctx, new = _plan_lengths(case)
    bs = case["block"]
    held = [_ceil(c, bs) for c in ctx]
    want = sum(max(0, _ceil(c + x, bs) - _ceil(c, bs)) for c, x in zip(ctx, new) if x > 0)
    free = int(want * case["spare"])
    num_blocks = sum(held) + free + 5
    max_blocks = max(_ceil(c + max(x, 0), bs) for c, x in zip(ctx, new)) + 1
    ids = torch.randperm(num_blocks, generator=g, device="cuda", dtype=torch.int32)
    held_t = _ints(held)
    col = torch.arange(max_blocks, device="cuda")
    at = (torch.cumsum(held_t, 0) - held_t)[:, None] + col[None]
    tables = torch.where(col[None] < held_t[:, None], ids[at.clamp(max=num_blocks - 1)], -1).to(torch.int32)
    ring = torch.full((num_blocks,), -1, dtype=torch.int32, device="cuda")
    head = int(torch.randint(num_blocks, (1,), generator=g, device="cuda"))
    ring[(head + torch.arange(free, device="cuda")) % num_blocks] = ids[sum(held):sum(held) + free]
    return dict(op="plan", context_lens=_ints(ctx), new_lens=_ints(new), block_tables=tables, free_ring=ring,
                ring_state=_ints([head, free]), block=bs, tokens=sum(max(x, 0) for x in new))


def _prepare_write(case, seed):
    g = _gen(seed)
    T, H, d, dt = case["tokens"], case["kv_heads"], case["d"], DTYPES[case["dtype"]]
    num_blocks = _ceil(T, case["block"]) + 3
    cache = lambda: torch.randn((num_blocks, case["block"], H, d), generator=g, device="cuda").to(dt)  # noqa: E731
    kc, vc = cache(), cache()
    # with `fused`, keys and values are slices of one projection that holds the queries too
    lead = 4 * H if case["fused"] else 0
    x = torch.randn((T, lead + 2 * H, d), generator=g, device="cuda").to(dt)
    k, v = (x[:, lead:lead + H], x[:, lead + H:]) if case["fused"] else (x[:, :H].contiguous(), x[:, H:].contiguous())
    slots = torch.randperm(num_blocks * case["block"], generator=g, device="cuda", dtype=torch.int32)[:T].contiguous()
    slots = torch.where(torch.rand(T, generator=g, device="cuda") < case["drop"], -1, slots).to(torch.int32)
    return dict(op="write", k=k, v=v, slot_map=slots, k_cache=kc, v_cache=vc)


def _attend_lengths(case):
    q = _lengths(case, case["q_lo"], case["q_hi"], 0)
    ctx = _lengths(case, case["ctx_lo"], case["ctx_hi"], 1)
    return q, [a + b for a, b in zip(q, ctx)]


def _prepare_attend(case, seed):
    g = _gen(seed)
    dt, bs, Hk, d = DTYPES[case["dtype"]], case["block"], case["kv_heads"], case["d"]
    q_lens, kv_lens = _attend_lengths(case)
    held = [_ceil(x, bs) for x in kv_lens]
    num_blocks, max_blocks, T = sum(held) + 3, max(held) + 1, sum(q_lens)
    ids = torch.randperm(num_blocks, generator=g, device="cuda", dtype=torch.int32)
    held_t, col = _ints(held), torch.arange(max_blocks, device="cuda")
    at = (torch.cumsum(held_t, 0) - held_t)[:, None] + col[None]
    tables = torch.where(col[None] < held_t[:, None], ids[at.clamp(max=num_blocks - 1)], -1).to(torch.int32)
    cache = lambda: torch.randn((num_blocks, bs, Hk, d), generator=g, device="cuda", dtype=dt)  # noqa: E731
    kc, vc = cache(), cache()
    # heads that look about and heads that look at few tokens
    sharp = torch.linspace(0.5, 3.0, case["heads"], device="cuda")[None, :, None]
    q = (torch.randn((T, case["heads"], d), generator=g, device="cuda") * sharp).to(dt)
    return dict(op="attend", q=q, k_cache=kc, v_cache=vc, block_tables=tables, seq_lens=_ints(kv_lens),
                cu_seqlens=_ints(_offsets(q_lens)), max_q_len=max(q_lens), max_seq_len=max(kv_lens),
                window=case["window"])


def _prepare_step(case, seed):
    g = _gen(seed)
    dt, H, Hk, dk, dv, N = (DTYPES[case["dtype"]], case["heads"], case["k_heads"], case["dk"], case["dv"],
                            case["n"])
    lens = _lengths(case, case["t_lo"], case["t_hi"], 0)
    T, slots = sum(lens), N + N // 4 + 2
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k, v = unit(rand(T, Hk, dk)).to(dt), unit(rand(T, Hk, dk)).to(dt), rand(T, H, dv).to(dt)
    beta = torch.sigmoid(rand(T, H))
    log_alpha = torch.nn.functional.logsigmoid(rand(T, H) + 2)
    pool = rand(slots, H, dv, dk) * 0.1
    index = torch.randperm(slots, generator=g, device="cuda", dtype=torch.int32)[:N].contiguous()
    old = torch.rand(N, generator=g, device="cuda") >= case["fresh"]
    return dict(op="step", q=q, k=k, v=v, log_alpha=log_alpha, beta=beta, state_pool=pool, state_index=index,
                cu_seqlens=_ints(_offsets(lens)), context_lens=torch.where(old, 100, 0).to(torch.int32),
                max_len=max(lens))


# ------------------------------------------------------------------ the passes --
def run(s):
    if own:
        return _run_own(s)
    return {"plan": _plain_plan, "write": _plain_write, "attend": _plain_attend, "step": _plain_step}[s["op"]](s)


def _run_own(s):
    import chunkwise_gated_deltanet_gb300 as gdn
    if s["op"] == "plan":
        p = gdn.paged_plan(s["context_lens"], s["new_lens"], s["block_tables"], s["free_ring"], s["ring_state"],
                           s["block"], s["tokens"])
        return dict(cu_seqlens=p.cu_seqlens, seq_lens=p.seq_lens, slot_map=p.slot_map, positions=p.positions,
                    granted=p.granted, ring_state=p.ring_state, block_tables=s["block_tables"],
                    free_ring=s["free_ring"])
    if s["op"] == "write":
        gdn.paged_write(s["k"], s["v"], s["slot_map"], s["k_cache"], s["v_cache"])
        return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    if s["op"] == "attend":
        out, lse = gdn.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["seq_lens"],
                                       s["cu_seqlens"], s["max_q_len"], max_seq_len=s["max_seq_len"],
                                       window=s["window"], return_lse=True)
        return dict(out=out, lse=lse)
    out = gdn.recurrent_step(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["state_pool"], s["state_index"],
                             s["cu_seqlens"], context_lens=s["context_lens"])
    return dict(out=out, state_pool=s["state_pool"])


def _plain_plan(s):
    ctx, new, tables, ring, bs = s["context_lens"], s["new_lens"], s["block_tables"], s["free_ring"], s["block"]
    (N, M), nb, dev = tables.shape, ring.numel(), ctx.device
    head, count = s["ring_state"][0], s["ring_state"][1]
    done, add = new < 0, new.clamp(min=0)
    old = (ctx + bs - 1) // bs
    fits = ctx + add <= M * bs
    need = torch.where(done | ~fits, 0, (ctx + add + bs - 1) // bs - old)
    cum = torch.cumsum(need, 0)
    granted = ~done & fits & ((need == 0) | (cum <= count))
    taken = torch.where(granted, need, 0).sum()
    col = torch.arange(M, device=dev)[None]
    # blocks of finished requests go to the ring's end, in row order
    back = done[:, None] & (col < old[:, None])
    rank = torch.cumsum(back.reshape(-1), 0) - 1
    at = torch.where(back.reshape(-1), (head + count + rank) % nb, nb)
    grown = torch.cat([ring, ring[:1]])
    fetched = ring[(head + (cum - need)[:, None] + col - old[:, None]) % nb]
    tables.copy_(torch.where(granted[:, None] & (col >= old[:, None]) & (col < (old + need)[:, None]), fetched, tables))
    grown[at] = tables.reshape(-1)
    ring.copy_(grown[:nb])
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(add, 0)])
    t = torch.arange(s["tokens"], device=dev)
    row = torch.searchsorted(cu[1:], t, right=True).clamp(max=N - 1)
    pos = ctx[row] + t - cu[row]
    inside = t < cu[-1]
    block = tables[row, (pos // bs).clamp(max=M - 1)]
    slot = torch.where(inside & granted[row], block * bs + pos % bs, -1)
    return dict(cu_seqlens=cu.int(), seq_lens=torch.where(granted, ctx + add, 0).int(), slot_map=slot.int(),
                positions=torch.where(inside, pos, -1).int(), granted=granted.int(),
                ring_state=torch.stack([(head + taken) % nb, count - taken + back.sum()]).int(), block_tables=tables,
                free_ring=ring)


def _plain_write(s):
    kc, vc, slots = s["k_cache"], s["v_cache"], s["slot_map"].long()
    there = slots >= 0
    kc.flatten(0, 1)[slots[there]] = s["k"][there]
    vc.flatten(0, 1)[slots[there]] = s["v"][there]
    return dict(k_cache=kc, v_cache=vc)


def _plain_attend(s):
    q, kc, vc, cu = s["q"], s["k_cache"], s["v_cache"], s["cu_seqlens"].long()
    T, H, d = q.shape
    bs, Hk = kc.shape[1], kc.shape[2]
    dev, L, S = q.device, s["max_q_len"], s["max_seq_len"]
    N = cu.numel() - 1
    kv_len, q_len = s["seq_lens"].long(), cu[1:] - cu[:-1]
    blocks = s["block_tables"][:, :(S + bs - 1) // bs].clamp(min=0).long()
    k = kc[blocks].flatten(1, 2)[:, :S].float()
    v = vc[blocks].flatten(1, 2)[:, :S].float()
    j = torch.arange(S, device=dev)
    v = torch.where((j[None] < kv_len[:, None])[..., None, None], v, 0.0)
    i = torch.arange(L, device=dev)
    rows = (cu[:-1, None] + i[None]).clamp(max=T - 1)
    qq = q[rows].float().view(N, L, Hk, H // Hk, d).permute(0, 2, 3, 1, 4).reshape(N, Hk, -1, d)
    pos = (kv_len - q_len)[:, None] + i[None]
    seen = j[None, None] <= pos[..., None]
    if s["window"]:
        seen &= j[None, None] > pos[..., None] - s["window"]
    seen &= (j[None] < kv_len[:, None])[:, None]
    x = (qq * d ** -0.5) @ k.permute(0, 2, 3, 1)
    x = x.view(N, Hk, H // Hk, L, S).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    safe = torch.where(torch.isinf(top), 0.0, top)
    x.sub_(safe).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (safe + torch.log(total))[..., 0]
    o = (x.view(N, Hk, -1, S) @ v.permute(0, 2, 1, 3)).view(N, Hk, H // Hk, L, d)
    o = torch.where(total > 0, o / total, 0.0)
    token = torch.arange(T, device=dev)
    n = torch.searchsorted(cu[1:], token, right=True).clamp(max=N - 1)
    at = token - cu[n]
    out = o.permute(0, 3, 1, 2, 4).reshape(N, L, H, d)[n, at].to(q.dtype)
    return dict(out=out, lse=lse.permute(0, 3, 1, 2).reshape(N, L, H)[n, at])


def _plain_step(s):
    """The chunk form of the recurrence with each request's tokens as one padded chunk."""
    v, pool, cu, L = s["v"], s["state_pool"], s["cu_seqlens"].long(), s["max_len"]
    T, H, dv = v.shape
    dk, Hk, N = s["k"].shape[-1], s["k"].shape[1], cu.numel() - 1
    dev = v.device
    i = torch.arange(L, device=dev)
    rows = (cu[:-1, None] + i[None]).clamp(max=T - 1)
    real = (i[None] < (cu[1:] - cu[:-1])[:, None])[..., None]
    pad = lambda x: torch.where(real[..., None], x[rows].float(), 0.0).transpose(1, 2)  # noqa: E731
    share = lambda x: x[:, :, None].expand(N, Hk, H // Hk, L, dk).reshape(N, H, L, dk)  # noqa: E731
    q, k, vv = share(pad(s["q"])), share(pad(s["k"])), pad(v)
    beta = torch.where(real, s["beta"][rows], 0.0).transpose(1, 2)
    gate = torch.where(real, s["log_alpha"][rows], 0.0).transpose(1, 2).cumsum(-1)
    slot = s["state_index"].long()
    S0 = torch.where((s["context_lens"] > 0)[:, None, None, None], pool[slot], 0.0)
    low = i[:, None] >= i[None]
    decay = torch.where(low, torch.exp(torch.where(low, gate[..., :, None] - gate[..., None, :], 0.0)), 0.0)
    kt = k.transpose(-1, -2)
    A = beta[..., None] * decay * (k @ kt)
    A = torch.where(i[:, None] > i[None], A, 0.0) + torch.eye(L, device=dev)
    eg = torch.exp(gate)[..., None]
    St = S0.transpose(-1, -2)
    u = torch.linalg.solve_triangular(A, beta[..., None] * (vv - eg * (k @ St)), upper=False, unitriangular=True)
    o = eg * (q @ St) + (decay * (q @ kt)) @ u
    last = gate[..., -1:]
    pool[slot] = torch.exp(last)[..., None] * S0 + (torch.exp(last - gate)[..., None] * u).transpose(-1, -2) @ k
    token = torch.arange(T, device=dev)
    n = torch.searchsorted(cu[1:], token, right=True).clamp(max=N - 1)
    return dict(out=o.transpose(1, 2)[n, token - cu[n]].to(v.dtype), state_pool=pool)


# ---------------------------------------------------------------- 64-bit values --
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": lambda c, s: None, "write": _exact_write, "attend": _exact_attend,
            "step": _exact_step}[case["op"]](case, s)


def _exact_write(case, s):
    kc, vc, bs = s["k_cache"].double(), s["v_cache"].double(), s["k_cache"].shape[1]
    for t, slot in enumerate(s["slot_map"].tolist()):
        if slot >= 0:
            kc[slot // bs, slot % bs] = s["k"][t].double()
            vc[slot // bs, slot % bs] = s["v"][t].double()
    return dict(k_cache=kc, v_cache=vc)


def _exact_attend(case, s):
    q, kc, vc, w = s["q"], s["k_cache"], s["v_cache"], s["window"]
    T, H, d = q.shape
    bs, G = kc.shape[1], H // kc.shape[2]
    q_lens, kv_lens = _attend_lengths(case)
    if sum(a * b for a, b in zip(q_lens, kv_lens)) * H * d * 4 > 1e13:
        return None
    out = torch.zeros((T, H, d), dtype=torch.float64, device=q.device)
    lse = torch.zeros((T, H), dtype=torch.float64, device=q.device)
    t0 = 0
    for n, (ql, kl) in enumerate(zip(q_lens, kv_lens)):
        held = s["block_tables"][n, :_ceil(kl, bs)].long()
        j = torch.arange(kl, device=q.device)
        p = torch.arange(kl - ql, kl, device=q.device)
        hide = j[None] > p[:, None]
        if w:
            hide |= j[None] <= p[:, None] - w
        k, v = kc[held].flatten(0, 1)[:kl], vc[held].flatten(0, 1)[:kl]
        # heads at a time, so that the scores take a bounded amount of memory
        step = max(1, min(H, int(4e8 / (ql * kl))))
        for h in range(0, H, step):
            kv = torch.arange(h, min(H, h + step), device=q.device) // G
            x = torch.einsum("ihd,jhd->hij", q[t0:t0 + ql, h:h + step].double(), k[:, kv].double()) / math.sqrt(d)
            x = x.masked_fill(hide, -math.inf)
            z = torch.logsumexp(x, -1)
            out[t0:t0 + ql, h:h + step] = torch.einsum("hij,jhd->ihd", torch.exp(x - z[..., None]), v[:, kv].double())
            lse[t0:t0 + ql, h:h + step] = z.T
        t0 += ql
    return dict(out=out, lse=lse)


def _exact_step(case, s):
    pool = s["state_pool"].double()
    T, H, dv = s["v"].shape
    out = torch.zeros((T, H, dv), dtype=torch.float64, device=pool.device)
    cu, ctx, slot = s["cu_seqlens"].tolist(), s["context_lens"].tolist(), s["state_index"].long()
    rep = H // s["k"].shape[1]
    S = pool[slot]
    for n, c in enumerate(ctx):
        if c == 0:
            S[n] = 0.0
    for t in range(max(b - a for a, b in zip(cu, cu[1:]))):
        act = [n for n in range(len(ctx)) if cu[n] + t < cu[n + 1]]
        tok = torch.tensor([cu[n] + t for n in act], device=pool.device)
        act = torch.tensor(act, device=pool.device)
        k, q = (s[x][tok].double().repeat_interleave(rep, 1) for x in ("k", "q"))
        v, a, b = s["v"][tok].double(), s["log_alpha"][tok].double().exp(), s["beta"][tok].double()
        M = a[..., None, None] * S[act]
        u = b[..., None] * (v - torch.einsum("nhvk,nhk->nhv", M, k))
        M = M + u[..., None] * k[..., None, :]
        out[tok] = torch.einsum("nhvk,nhk->nhv", M, q)
        S[act] = M
    pool[slot] = S
    return dict(out=out, state_pool=pool)


# ------------------------------------------------------------------- the floors --
def work(case):
    op = case["op"]
    if op == "plan":
        ctx, new = _plan_lengths(case)
        bs, N = case["block"], case["n"]
        grown = sum(max(0, _ceil(c + x, bs) - _ceil(c, bs)) for c, x in zip(ctx, new) if x > 0)
        back = sum(_ceil(c, bs) for c, x in zip(ctx, new) if x < 0)
        T = sum(max(x, 0) for x in new)
        # lengths in; offsets, lengths and grants out; slots and positions; ring entries read or
        # written with the table entries they come from or go to
        return {"bytes": 4.0 * (2 * N + 3 * N + 1 + 2 * T + 2 * grown + 2 * back + 4), "flops": 0.0}
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "write":
        return {"bytes": case["tokens"] * (4.0 * case["kv_heads"] * case["d"] * size + 4), "flops": 0.0}
    if op == "attend":
        q_lens, kv_lens = _attend_lengths(case)
        pairs, read = 0, 0
        w = case["window"] or 1 << 60
        for a, b in zip(q_lens, kv_lens):
            first = b - a + 1  # keys that the first new token sees, without a window
            full = max(0, min(a, b - w + 1)) if w >= first else a
            pairs += full * w if w < 1 << 60 else 0
            ramp = a - full if w < 1 << 60 else a
            pairs += ramp * first + ramp * (ramp - 1) // 2
            read += min(b, w + a - 1)
        rows = sum(q_lens) * case["heads"]
        return {"bytes": float(read * case["kv_heads"] * case["d"] * 2 * size + rows * (case["d"] * 2 * size + 4)),
                "flops": 4.0 * case["d"] * case["heads"] * pairs}
    lens = _lengths(case, case["t_lo"], case["t_hi"], 0)
    T, N, H, dk, dv = sum(lens), case["n"], case["heads"], case["dk"], case["dv"]
    old = N * (1 - case["fresh"])
    return {"bytes": (N + old) * H * dk * dv * 4.0
            + T * (2.0 * case["k_heads"] * dk * size + 2 * H * dv * size + 8 * H),
            "flops": 8.0 * T * H * dk * dv}
