"""The serving operators on the GPU against plain 64-bit references (tests/serving_ref.py,
which derives the attention's error bounds) and, for the recurrence, the oracle.

Recurrence: fp32 arithmetic from inputs that fp64 holds exactly, so the states take the
fp32 bound max|delta| / max|ref| <= 1e-4 for both dtypes; outputs the same, plus their own
storage rounding, 2^-8 |ref|, in bf16.
"""
import math

import numpy as np
import pytest
import torch

import chunkwise_gated_deltanet_gb300 as gdn
from oracle import native
from tests import serving_ref as R
from tests.parity import TOL_F32_REL_MAX

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_gated_deltanet_gb300 import build
    build.build()
    gdn.load_library()


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------- plan --
def _plan_inputs(N, block, ctx_hi, new_hi, ended, spare, seed):
    r = np.random.RandomState(seed)
    ctx = r.randint(0, ctx_hi + 1, N)
    new = np.where(r.rand(N) < ended, -1, r.randint(0, new_hi + 1, N))
    held = -(-ctx // block)
    want = int(sum(max(0, -(-(c + x) // block) - -(-c // block)) for c, x in zip(ctx, new) if x > 0))
    free = int(want * spare)
    nb = int(held.sum()) + free + 3
    M = int(max([-(-(c + max(x, 0)) // block) for c, x in zip(ctx, new)] + [1]))
    ids = r.permutation(nb)
    tables = np.full((N, M), -1)
    at = 0
    for n in range(N):
        tables[n, :held[n]] = ids[at:at + held[n]]
        at += held[n]
    ring = np.full(nb, -1)
    head = int(r.randint(nb))
    for i in range(free):
        ring[(head + i) % nb] = ids[at + i]
    return ctx, new, tables, ring, np.array([head, free])


def _run_plan(ctx, new, tables, ring, state, block, T):
    t, f = _i32(tables), _i32(ring)
    p = gdn.paged_plan(_i32(ctx), _i32(new), t, f, _i32(state), block, T)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in p._asdict().items()}
    got.update(block_tables=t.cpu().numpy(), free_ring=f.cpu().numpy())
    return got


@pytest.mark.parametrize("N,block,ctx_hi,new_hi,ended,spare", [
    (1, 16, 0, 1, 0.0, 1.0), (1, 8, 40, 0, 0.0, 1.0), (7, 16, 100, 1, 0.0, 1.0),
    (300, 24, 500, 70, 0.2, 1.0), (2049, 16, 60, 9, 0.3, 0.5), (4500, 8, 20, 3, 0.1, 2.0),
    (5, 128, 5000, 3000, 0.0, 1.0), (64, 1024, 5000, 10, 0.5, 1.0)])
@pytest.mark.parametrize("room", [0, 11, -5])
def test_plan_equals_the_plain_form(N, block, ctx_hi, new_hi, ended, spare, room):
    """Whole numbers, so equal: with room for more tokens than there are, and for fewer."""
    args = _plan_inputs(N, block, ctx_hi, new_hi, ended, spare, seed=N + block)
    T = max(0, int(np.maximum(args[1], 0).sum()) + room)
    got, ref = _run_plan(*args, block, T), R.plan(*args, block, T)
    for name, want in ref.items():
        assert np.array_equal(got[name], want), name


def test_plan_refuses_what_does_not_fit():
    """A request past its table row is refused without taking blocks; one past the free
    blocks is refused and so are later ones that need any, but not those that need none."""
    block, M = 8, 3
    ctx, new = np.array([16, 5, 8, 7, 0]), np.array([9, 4, 16, 1, 1])
    tables = np.full((5, M), -1)
    tables[0, :2], tables[1, 0], tables[2, 0], tables[3, 0] = [4, 5], 6, 7, 8
    ring = np.array([0, 1, -1, -1, -1, -1, -1, -1, -1, -1])
    got = _run_plan(ctx, new, tables, ring, np.array([0, 2]), block, 31)
    assert got["granted"].tolist() == [0, 1, 0, 1, 0]
    assert got["seq_lens"].tolist() == [0, 9, 0, 8, 0]
    assert got["ring_state"].tolist() == [1, 1]
    assert got["block_tables"][1].tolist() == [6, 0, -1] and got["block_tables"][2].tolist() == [7, -1, -1]
    assert (got["slot_map"][:9] == -1).all() and got["slot_map"][9:13].tolist() == [53, 54, 55, 0]
    ref = R.plan(ctx, new, tables, ring, np.array([0, 2]), block, 31)
    for name, want in ref.items():
        assert np.array_equal(got[name], want), name


def test_plan_recycles_over_many_steps():
    """Requests come, grow, end and come again: blocks are never held twice or lost."""
    r = np.random.RandomState(0)
    N, block, M, nb = 40, 8, 12, 300
    tables, ring, state = _i32(np.full((N, M), -1)), _i32(np.arange(nb)), _i32([0, nb])
    ctx = np.zeros(N, int)
    for step in range(60):
        new = np.where((ctx > 60) & (r.rand(N) < 0.5), -1, np.where(ctx == 0, r.randint(0, 30, N), 1))
        new = np.where((new > 0) & (ctx + new > M * block), 0, new)
        p = gdn.paged_plan(_i32(ctx), _i32(new), tables, ring, state, block, int(np.maximum(new, 0).sum()))
        state = p.ring_state
        seq, ok = p.seq_lens.cpu().numpy(), p.granted.cpu().numpy()
        ctx = np.where(new < 0, 0, np.where(ok > 0, seq, ctx))
        held = [int(x) for n in range(N) for x in tables[n, :-(-ctx[n] // block)].cpu()]
        head, count = (int(x) for x in state.cpu())
        free = [int(ring[(head + i) % nb]) for i in range(count)]
        assert sorted(held + free) == list(range(nb)), step


def test_plan_without_requests_and_with_broken_state():
    z = np.zeros(0, int)
    got = _run_plan(z, z, np.zeros((0, 4), int), np.arange(5), np.array([3, 2]), 16, 6)
    assert got["cu_seqlens"].tolist() == [0] and got["ring_state"].tolist() == [3, 2]
    assert (got["slot_map"] == -1).all() and (got["positions"] == -1).all()
    # lengths and ring state out of range: in bounds, slots only where blocks are real
    got = _run_plan(np.array([-3, 2 ** 31 - 1, 5]), np.array([4, 5, 2 ** 31 - 1]),
                    np.array([[99], [-5], [1]]), np.array([77, -1, 2]), np.array([-4, 100]), 8, 20)
    assert got["granted"].tolist() == [1, 0, 0]
    # ring position -4 mod 3 = 2 holds block 2
    assert got["slot_map"][:4].tolist() == [16, 17, 18, 19] and (got["slot_map"][4:] == -1).all()


# ------------------------------------------------------------------------ write --
@pytest.mark.parametrize("T,H,d,block", [(1, 1, 16, 8), (37, 3, 128, 16), (1000, 8, 64, 24), (0, 2, 32, 8),
                                         (513, 5, 32, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fused", [False, True])
def test_write_moves_rows_to_their_slots(T, H, d, block, dtype, fused):
    g = torch.Generator().manual_seed(T + d)
    nb, dt = T // block + 4, DT[dtype]
    kc, vc = (torch.randn(nb, block, H, d, generator=g).to(dt) for _ in range(2))
    x = torch.randn(T, 2 * H + 3, d, generator=g).to(dt)
    slots = torch.randperm(nb * block, generator=g)[:T].to(torch.int32)
    slots[::7] = -1
    if T > 3:
        slots[3] = nb * block  # out of range: passed over
    want_k, want_v = kc.clone(), vc.clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < nb * block:
            want_k[s // block, s % block], want_v[s // block, s % block] = x[t, 3:3 + H], x[t, 3 + H:]
    xd = x.to(DEV)
    k, v = xd[:, 3:3 + H], xd[:, 3 + H:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    kd, vd = kc.to(DEV), vc.to(DEV)
    gdn.paged_write(k, v, slots.to(DEV), kd, vd)
    assert torch.equal(kd.cpu(), want_k) and torch.equal(vd.cpu(), want_v)


# -------------------------------------------------------------------- attention --
def _attend(q_lens, kv_lens, Hq, Hkv, d, block, dtype, window=0, seed=0, q_pad=0, edit=None,
            max_seq_len=None, scale=None, sharp=2.0):
    """Runs the operator and the reference; edit(n, k, v) changes a request's keys and
    values (in the pages too).  Returns per request (out, lse, reference tuple)."""
    dt = DT[dtype]
    kc, vc, tables, keys, values = R.pages(kv_lens, Hkv, d, block, dt, seed, DEV)
    if edit:
        for n, x in enumerate(kv_lens):
            edit(n, keys[n], values[n])
            for j in range(x):
                b = int(tables[n, j // block])
                kc[b, j % block], vc[b, j % block] = keys[n][j].to(DEV), values[n][j].to(DEV)
    T = sum(q_lens)
    g = torch.Generator().manual_seed(seed + 1)
    wide = (torch.randn(T, Hq + q_pad, d, generator=g) * sharp).to(dt).to(DEV)
    q = wide[:, :Hq]
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    out, lse = gdn.paged_attention(q, kc, vc, tables, _i32(kv_lens), _i32(cu), max(q_lens + [0]),
                                   max_seq_len=max(kv_lens + [0]) if max_seq_len is None else max_seq_len,
                                   window=window, scale=scale, return_lse=True)
    gdn.gdn_check_status()
    torch.cuda.synchronize()
    res = []
    for n in range(len(q_lens)):
        sl = slice(cu[n], cu[n + 1])
        ref = R.attention(q[sl], keys[n], values[n], kv_lens[n] - q_lens[n],
                          d ** -0.5 if scale is None else scale, window)
        res.append((out[sl].double().cpu(), lse[sl].double().cpu(), ref))
    return res


def _check_attend(res, d, kv_lens, bf16, what=""):
    for n, (o, z, (ro, rz, A, X)) in enumerate(res):
        empty = torch.isinf(rz)
        assert (z[empty] == -math.inf).all() and (o[empty] == 0).all(), f"{what} request {n}: empty rows"
        to, tz = R.bounds(ro, torch.where(empty, 0.0, rz), A, X, d, kv_lens[n], bf16)
        assert torch.isfinite(o).all() and torch.isfinite(z[~empty]).all(), f"{what} request {n}"
        assert ((o - ro).abs() <= to).all(), f"{what} request {n}: out {((o - ro).abs() - to).max()}"
        assert ((z - rz).abs()[~empty] <= tz[~empty]).all(), f"{what} request {n}: lse"


SHAPES = [(16, 4, 128), (8, 8, 64), (6, 2, 128), (5, 1, 64), (4, 2, 32), (2, 1, 16), (32, 1, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
def test_attention_one_token(Hq, Hkv, d, dtype):
    """Decoding: lengths of one, around tile and page edges, and of zero."""
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 0]
    res = _attend([1] * len(kv), kv, Hq, Hkv, d, 16, dtype, seed=d)
    _check_attend(res, d, kv, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
def test_attention_ragged_chunks(Hq, Hkv, d, dtype):
    """Chunks of new tokens: none, one, more than the sequence holds, past a row block."""
    ql, kv = [0, 1, 5, 70, 3, 33, 9], [40, 1, 133, 70, 0, 200, 4]
    res = _attend(ql, kv, Hq, Hkv, d, 16, dtype, seed=d + 1, q_pad=3)
    _check_attend(res, d, kv, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [8, 16, 24, 48, 64, 128, 200, 256, 1024])
def test_attention_page_sizes(block, d, dtype):
    ql, kv = [7, 1, 40], [131, 257, 90]
    res = _attend(ql, kv, 4, 2, d, block, dtype, seed=block)
    _check_attend(res, d, kv, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 100, 1000])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_window(window, d, dtype):
    ql, kv = [1, 90, 6, 1], [300, 200, 260, 64]
    res = _attend(ql, kv, 8, 2, d, 16, dtype, window=window, seed=window)
    _check_attend(res, d, kv, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,ql", [(128, 1), (128, 3), (64, 1), (128, 40)])
def test_attention_long_axis_is_split(d, ql, dtype):
    """Few rows over a long cache: shared by many CTAs and joined."""
    kv = [9001, 3]
    res = _attend([ql, 1], kv, 4, 1, d, 64, dtype, seed=ql)
    _check_attend(res, d, kv, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_many_row_blocks(dtype):
    """Whole prompts: several row blocks a request, causal from the first token on."""
    ql, kv = [300, 129, 64], [300, 129, 64]
    res = _attend(ql, kv, 6, 2, 128, 16, dtype, seed=3)
    _check_attend(res, 128, kv, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_many_requests(dtype):
    """More requests than one launch schedules."""
    r = np.random.RandomState(1)
    ql, kv = [int(x) for x in r.randint(0, 3, 1300)], [int(x) for x in r.randint(0, 40, 1300)]
    res = _attend(ql, kv, 2, 1, 64, 8, dtype, seed=4)
    _check_attend(res, 64, kv, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,sharp", [(1.0, 0.02), (0.3, 30.0), (1e-6, 1.0)])
def test_attention_scales(scale, sharp, dtype):
    """Nearly uniform and nearly one-hot rows."""
    ql, kv = [2, 70], [150, 500]
    res = _attend(ql, kv, 4, 2, 128, 16, dtype, scale=scale, sharp=sharp, seed=9)
    _check_attend(res, 128, kv, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ql,kv", [(4, 100), (60, 160), (300, 300)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attention_masked_tokens_do_not_reach_others(ql, kv, bad, dtype):
    """A non-finite key or value of a later token, or of one before the window, reaches the
    tokens that see it and no others."""
    def edit(n, k, v):
        k[kv - 1], v[kv - 2, :, 5] = bad, bad
        k[0], v[1] = bad, bad
    w = kv - ql if kv > ql else 0
    res = _attend([ql], [kv], 4, 2, 128, 16, dtype, window=w, edit=edit, seed=5)
    o, z, (ro, rz, A, X) = res[0]
    p = kv - ql + torch.arange(ql)
    first = torch.clamp(p - w + 1, min=0) if w else torch.zeros(ql, dtype=torch.int64)
    clean = (p < kv - 2) & (first > 1)
    if w:
        assert clean.any()
    part = lambda x: x[clean]  # noqa: E731
    _check_attend([(part(o), part(z), tuple(part(x) for x in (ro, rz, A, X)))], 128, [kv], dtype == "bf16")
    # the value's column alone, for a row that sees the bad value and no bad key
    row = ql - 2
    if w and int(first[row]) > 1:
        assert not torch.isfinite(o[row, :, 5]).any()
        assert torch.isfinite(o[row][:, [c for c in range(128) if c != 5]]).all()
    assert torch.isfinite(z[clean]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_bad_inputs_stay_in_bounds(dtype):
    """Offsets, lengths and table entries out of range give defined results."""
    dt = DT[dtype]
    kc, vc, tables, keys, values = R.pages([40, 40], 2, 64, 8, dt, 0, DEV)
    q = torch.randn(6, 4, 64, device=DEV).to(dt)
    out = torch.full((6, 4, 64), 7.0, device=DEV, dtype=dt)
    lse = torch.full((6, 4), 7.0, device=DEV)
    ws = torch.empty(gdn.gdn_paged_attention_workspace_bytes(4, 2, 64, 3, dt), dtype=torch.uint8, device=DEV)
    gdn.gdn_paged_attention(q, kc, vc, tables, _i32([2 ** 31 - 1, -5]), _i32([-3, 2, 2 ** 31 - 1]), out, lse, ws, 3)
    torch.cuda.synchronize()
    gdn.gdn_check_status()
    assert (lse[2:] == -math.inf).all() and (out[2:] == 0).all()  # length below 0: empty
    out.fill_(7.0)
    gdn.gdn_paged_attention(q, kc, vc, tables, _i32([40, 40]), _i32([1, 3, 2]), out, lse, ws, 3)
    torch.cuda.synchronize()
    assert (out[0] == 7).all() and (out[3:] == 7).all() and not (out[1:3] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_same_bits_again_and_on_another_stream(dtype):
    ql, kv = [1, 17, 260], [2000, 700, 900]
    dt = DT[dtype]
    kc, vc, tables, _, _ = R.pages(kv, 2, 128, 16, dt, 3, DEV)
    q = torch.randn(sum(ql), 8, 128, device=DEV).to(dt)
    cu, sl = _i32(np.concatenate([[0], np.cumsum(ql)])), _i32(kv)
    a = gdn.paged_attention(q, kc, vc, tables, sl, cu, 260, return_lse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = gdn.paged_attention(q, kc, vc, tables, sl, cu, 260, return_lse=True)
    s.synchronize()
    # neither hint changes a value's meaning
    c = gdn.paged_attention(q, kc, vc, tables, sl, cu, 5000, max_seq_len=1 << 20, return_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (a[1] - c[1]).abs().max() < 1e-4


# -------------------------------------------------------------------- recurrence --
def _step_inputs(lens, Hk, H, dk, dv, dtype, seed, fresh=()):
    g = torch.Generator().manual_seed(seed)
    T, N, dt = sum(lens), len(lens), DT[dtype]
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = (unit(torch.randn(T, Hk, dk, generator=g)).to(dt) for _ in range(2))
    v = torch.randn(T, H, dv, generator=g).to(dt)
    beta = torch.sigmoid(torch.randn(T, H, generator=g))
    la = torch.nn.functional.logsigmoid(torch.randn(T, H, generator=g) + 2)
    pool = torch.randn(N + 3, H, dv, dk, generator=g) * 0.1
    index = torch.randperm(N + 3, generator=g)[:N].to(torch.int32)
    ctx = torch.tensor([0 if n in fresh else 9 for n in range(N)], dtype=torch.int32)
    return q, k, v, la, beta, pool, index, ctx


def _check_step(lens, Hk, H, dk, dv, dtype, seed=0, fresh=(), pad=0, use_ctx=True):
    q, k, v, la, beta, pool, index, ctx = _step_inputs(lens, Hk, H, dk, dv, dtype, seed, fresh)
    for n in fresh:
        pool[index[n]] = math.nan  # a new request's slot holds anything
    d = [x.to(DEV) for x in (q, k, v)]
    if pad:
        wide = [torch.cat([x, torch.zeros(x.shape[0], pad, x.shape[2], dtype=x.dtype, device=DEV)], 1) for x in d]
        d = [w[:, :x.shape[1]] for w, x in zip(wide, d)]
    cu = np.concatenate([[0], np.cumsum(lens)])
    pd = pool.to(DEV)
    out = gdn.recurrent_step(*d, la.to(DEV), beta.to(DEV), pd, index.to(DEV), _i32(cu),
                             context_lens=ctx.to(DEV) if use_ctx else None)
    torch.cuda.synchronize()
    out, after = out.double().cpu().numpy(), pd.double().cpu().numpy()
    want = pool.double().numpy().copy()
    ref = np.zeros(out.shape)
    rep = H // Hk
    for n, L in enumerate(lens):
        if L == 0:
            continue
        sl = slice(cu[n], cu[n + 1])
        S0 = torch.zeros(1, H, dv, dk) if n in fresh else pool[index[n]][None]
        o, S = native.gdn_forward_c(q[None, sl].repeat_interleave(rep, 2).contiguous(),
                                    k[None, sl].repeat_interleave(rep, 2).contiguous(), v[None, sl].contiguous(),
                                    la[None, sl].contiguous(), beta[None, sl].contiguous(), S0.contiguous(), None)
        ref[sl], want[int(index[n])] = o[0], S[0]
    live = np.isfinite(want)
    assert np.array_equal(live, np.isfinite(after))
    scale = np.abs(want[live]).max()
    assert np.abs(after[live] - want[live]).max() <= TOL_F32_REL_MAX * scale
    if sum(lens):
        slack = 2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0
        assert (np.abs(out - ref) - slack).max() <= TOL_F32_REL_MAX * np.abs(ref).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (32, 32), (16, 16), (16, 128), (128, 16), (64, 32), (32, 64)])
def test_step_matches_the_oracle(dk, dv, dtype):
    _check_step([1, 3, 0, 8, 9, 17, 1], 2, 4, dk, dv, dtype, seed=dk + dv, fresh=(1, 2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [1] * 33, [130, 64, 1], [2, 2, 2, 2, 2]])
def test_step_lengths(lens, dtype):
    _check_step(lens, 4, 4, 128, 128, dtype, seed=len(lens), pad=2, use_ctx=False)


def test_step_shared_key_heads_and_no_tokens():
    _check_step([5, 2], 1, 8, 64, 64, "bf16", seed=3)
    _check_step([5, 2], 3, 6, 64, 64, "f32", seed=4, fresh=(0,))
    _check_step([0, 0], 2, 2, 64, 64, "f32", seed=5, fresh=(0,))


def test_step_gates_at_their_ends():
    """alpha = 1, alpha = 0 (log alpha = -inf), beta = 0 and beta = 1."""
    q, k, v, la, beta, pool, index, ctx = _step_inputs([4, 4, 4], 2, 2, 64, 64, "f32", 6)
    la[0], la[2], beta[5], beta[9] = 0.0, -math.inf, 0.0, 1.0
    pd = pool.to(DEV)
    out = gdn.recurrent_step(*(x.to(DEV) for x in (q, k, v, la, beta)), pd, index.to(DEV), _i32([0, 4, 8, 12]))
    for n in range(3):
        sl = slice(4 * n, 4 * n + 4)
        S = pool[index[n]].double()
        for t in range(sl.start, sl.stop):
            a, b = la[t].double().exp()[:, None, None], beta[t].double()[:, None]
            u = b * (v[t].double() - torch.einsum("hvk,hk->hv", a * S, k[t].double()))
            S = a * S + u[:, :, None] * k[t].double()[:, None]
            o = torch.einsum("hvk,hk->hv", S, q[t].double())
            assert (out[t].double().cpu() - o).abs().max() < 1e-5
        assert (pd[index[n]].double().cpu() - S).abs().max() < 1e-5


def test_step_passes_over_slots_out_of_range_and_equals_decode():
    q, k, v, la, beta, pool, index, _ = _step_inputs([1, 1, 1, 1], 2, 2, 128, 128, "bf16", 7)
    index[1], index[2] = -1, pool.shape[0]
    pd = pool.to(DEV)
    d = [x.to(DEV) for x in (q, k, v, la, beta)]
    out = gdn.recurrent_step(*d, pd, index.to(DEV), _i32([0, 1, 2, 3, 4]))
    assert (out[1:3] == 0).all()
    S = pool[index[[0, 3]].long()].to(DEV)
    rows = torch.tensor([0, 3], device=DEV)
    o = gdn.decode_step(*(x[rows].contiguous() for x in d), S)
    assert (o.float() - out[rows].float()).abs().max() <= 2.0 ** -7 * o.float().abs().max()
    assert (S - pd[index[[0, 3]].long()]).abs().max() < 1e-5
    untouched = [i for i in range(pool.shape[0]) if i not in (int(index[0]), int(index[3]))]
    assert torch.equal(pd.cpu()[untouched], pool[untouched])


def test_step_continues_the_chunk_forward():
    """A prompt through gdn_chunk_fwd, its final states put into the pool, then a few tokens
    at once: equal to one run over all tokens."""
    q, k, v, la, beta, pool, index, _ = _step_inputs([75], 2, 2, 64, 64, "f32", 8)
    d = [x.to(DEV) for x in (q, k, v, la, beta)]
    full, Sf = gdn.chunk_fwd(*(x[None] for x in d))
    _, S0 = gdn.chunk_fwd(*(x[None, :70].contiguous() for x in d))
    pd = pool.to(DEV)
    pd[int(index[0])] = S0[0]
    out = gdn.recurrent_step(*(x[70:] for x in d), pd, index.to(DEV), _i32([0, 5]))
    assert (out - full[0, 70:]).abs().max() <= 1e-4 * full.abs().max()
    assert (pd[int(index[0])] - Sf[0]).abs().max() <= 1e-4 * Sf.abs().max()


@pytest.mark.parametrize("d,ql,kv", [(128, 9, 9001), (64, 7, 5000), (128, 32, 129), (128, 5, 128), (64, 20, 2500)])
def test_attention_units_of_up_to_128_rows(d, ql, kv):
    """17 to 128 rows a key/value head: both halves of the tensor-core kernel take the same
    rows, over one tile, a few, and a split axis."""
    lens = [kv, 300, ql]
    res = _attend([ql, 6, ql], lens, 4, 1, d, 16, "bf16", seed=ql)
    _check_attend(res, d, lens, True)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attention_masked_tokens_in_small_units(bad):
    """The same as for whole row blocks: a bad value of a late token, 36 rows over 3 tiles."""
    ql, kv = 9, 300

    def edit(n, k, v):
        v[kv - 4, :, 7] = bad
    o, z, (ro, rz, A, X) = _attend([ql], [kv], 4, 1, 128, 16, "bf16", edit=edit, seed=2)[0]
    sees = kv - ql + torch.arange(ql) >= kv - 4
    assert not torch.isfinite(o[sees][:, :, 7]).any()
    part = lambda x: x[~sees]  # noqa: E731
    _check_attend([(part(o), part(z), tuple(part(x) for x in (ro, rz, A, X)))], 128, [kv], True)
    cols = [c for c in range(128) if c != 7]
    to, _ = R.bounds(ro, rz, A, X, 128, kv, True)
    assert ((o - ro).abs() <= to)[:, :, cols].all()


def test_attention_caches_beyond_l2():
    """Keys and values that pass half of L2, several waves of row blocks: a sample of rows."""
    ql, kv, Hq, Hkv, d, block = [1300, 700], [17000, 9000], 64, 8, 128, 32
    g = torch.Generator(device=DEV).manual_seed(0)
    held = [-(-x // block) for x in kv]
    nb = sum(held)
    ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    tables = torch.full((2, max(held)), -1, dtype=torch.int32, device=DEV)
    tables[0, :held[0]], tables[1, :held[1]] = ids[:held[0]], ids[held[0]:]
    kc, vc = (torch.randn(nb, block, Hkv, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(sum(ql), Hq, d, generator=g, device=DEV).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(ql)])
    out, lse = gdn.paged_attention(q, kc, vc, tables, _i32(kv), _i32(cu), max(ql), return_lse=True)
    gdn.gdn_check_status()
    r = np.random.RandomState(0)
    for n in range(2):
        k = kc[tables[n, :held[n]].long()].flatten(0, 1)[:kv[n]]
        v = vc[tables[n, :held[n]].long()].flatten(0, 1)[:kv[n]]
        rows = sorted(set(r.randint(0, ql[n], 40)) | {0, ql[n] - 1})
        for i in rows:
            h = int(r.randint(Hq))
            p = kv[n] - ql[n] + i
            kk, vv = k[:p + 1, h * Hkv // Hq][:, None], v[:p + 1, h * Hkv // Hq][:, None]
            ref = R.attention(q[cu[n] + i, h][None, None], kk, vv, p, d ** -0.5, 0)
            got = (out[cu[n] + i, h].double().cpu()[None, None], lse[cu[n] + i, h].double().cpu()[None, None], ref)
            _check_attend([got], d, [kv[n]], True, f"token {i} head {h}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_bad_tokens_reach_later_ones_only(dtype):
    """A non-finite value of one token leaves the tokens before it, the other rows and the other
    requests as they are."""
    q, k, v, la, beta, pool, index, _ = _step_inputs([7, 3], 2, 2, 64, 64, dtype, 11)
    run = lambda v, k: gdn.recurrent_step(  # noqa: E731
        *(x.to(DEV) for x in (q, k, v, la, beta)), pool.to(DEV), index.to(DEV), _i32([0, 7, 10]))
    good = run(v, k)
    v2, k2 = v.clone(), k.clone()
    v2[4, 0, 5] = math.inf
    bad = run(v2, k2)
    assert not torch.isfinite(bad[4:7, 0, 5]).any()
    bad[4:7, 0, 5] = good[4:7, 0, 5]
    assert torch.equal(bad, good)
    k2[5, 1] = math.nan
    bad = run(v, k2)
    assert torch.equal(bad[:5], good[:5]) and torch.equal(bad[7:], good[7:]) and torch.equal(bad[:, 0], good[:, 0])
    assert torch.isnan(bad[5:7, 1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("most", [3, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_step_more_units_than_the_gpu_holds(d, most, dtype):
    """Requests without tokens, new ones and slots out of range in between, token by token and
    in chunks; 800 (request, head) pairs."""
    N, H = 200, 4
    g = torch.Generator().manual_seed(most + d)
    lens = torch.randint(0, most + 1, (N,), generator=g).tolist()
    q, k, v, la, beta, pool, index, ctx = _step_inputs(lens, 2, H, d, d, dtype, 21, fresh=range(0, N, 7))
    gone = list(range(3, N, 11))
    index[gone[::2]], index[gone[1::2]] = -1, pool.shape[0]
    cu = np.concatenate([[0], np.cumsum(lens)])
    pd = pool.to(DEV)
    out = gdn.recurrent_step(*(x.to(DEV) for x in (q, k, v, la, beta)), pd, index.to(DEV), _i32(cu),
                             context_lens=ctx.to(DEV)).double().cpu().numpy()
    want, ref = pool.double().numpy().copy(), np.zeros(out.shape)
    for n, L in enumerate(lens):
        if L == 0 or n in gone:
            continue
        sl = slice(cu[n], cu[n + 1])
        S0 = pool[index[n]][None] * float(ctx[n] > 0)
        o, S = native.gdn_forward_c(q[None, sl].repeat_interleave(2, 2).contiguous(),
                                    k[None, sl].repeat_interleave(2, 2).contiguous(), v[None, sl].contiguous(),
                                    la[None, sl].contiguous(), beta[None, sl].contiguous(), S0.contiguous(), None)
        ref[sl], want[int(index[n])] = o[0], S[0]
    slack = 2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0
    assert (np.abs(out - ref) - slack).max() <= TOL_F32_REL_MAX * np.abs(ref).max()
    assert np.abs(pd.double().cpu().numpy() - want).max() <= TOL_F32_REL_MAX * np.abs(want).max()
    for n in gone:
        assert (out[cu[n]:cu[n + 1]] == 0).all()
    still = [int(index[n]) for n in range(N) if lens[n] == 0 and n not in gone]
    assert torch.equal(pd.cpu()[still], pool[still])


@pytest.mark.parametrize("lens", [[3, 1, 0, 6], [40, 17]])
def test_plan_write_and_step_on_another_stream(lens):
    """Inputs that a side stream is still writing when the calls are made on it."""
    N, T, bs = len(lens), sum(lens), 16
    q, k, v, la, beta, pool, index, _ = _step_inputs(lens, 2, 2, 64, 64, "bf16", 31)
    host = [x.pin_memory() for x in (q, k, v, la, beta, pool, index)]
    cu, new = _i32(np.concatenate([[0], np.cumsum(lens)])), torch.tensor(lens, dtype=torch.int32).pin_memory()

    def run(stream):
        tables = torch.full((N, 4), -1, dtype=torch.int32, device=DEV)
        ring, ctx = torch.arange(16, dtype=torch.int32, device=DEV), torch.zeros(N, dtype=torch.int32, device=DEV)
        state = _i32([0, 16])
        caches = [torch.zeros(16, bs, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        d = [torch.zeros_like(x, device=DEV) for x in host]
        n = torch.zeros(N, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            torch.cuda._sleep(2_000_000)
            for x, h in zip(d + [n], host + [new]):
                x.copy_(h, non_blocking=True)
            p = gdn.paged_plan(ctx, n, tables, ring, state, bs, T)
            gdn.paged_write(d[1], d[1], p.slot_map, *caches)
            out = gdn.recurrent_step(*d[:5], d[5], d[6], p.cu_seqlens, context_lens=ctx)
        stream.synchronize()
        assert torch.equal(p.cu_seqlens, cu)
        return [*p, tables, ring, *caches, out, d[5]]

    for a, b in zip(run(torch.cuda.current_stream()), run(torch.cuda.Stream())):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ql,kv", [(3, 500), (7, 200), (8, 2000), (13, 700), (30, 700), (100, 800)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attention_values_that_all_rows_see(ql, kv, bad, dtype):
    """A non-finite value in a tile that every row sees whole: its column gets it, from 12 rows
    to several row blocks; the other columns are as without it."""
    def edit(n, k, v):
        v[9, :, 7] = bad
    o, z, (ro, rz, A, X) = _attend([ql], [kv], 4, 1, 128, 16, dtype, edit=edit, seed=ql)[0]
    got = o[:, :, 7]
    assert torch.isnan(got).all() if math.isnan(bad) else (got == bad).all()
    cols = [c for c in range(128) if c != 7]
    to, tz = R.bounds(ro, rz, A, X, 128, kv, dtype == "bf16")
    assert ((o - ro).abs() <= to)[:, :, cols].all() and ((z - rz).abs() <= tz).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,ql,kv,window", [(8, 4, 5000, 0), (8, 4, 130, 0), (4, 8, 8, 0), (8, 3, 100, 7),
                                            (4, 16, 3001, 0), (8, 8, 128, 0), (8, 7, 1000, 200), (16, 2, 33, 0)])
def test_attention_units_of_up_to_64_rows(g, ql, kv, window, d):
    """Units that the tensor-core kernel holds in 2 or 4 copies, whole and split, with rows that
    see nothing in some copies' columns."""
    q_lens, kv_lens = [ql, ql, 1, ql - 1], [kv, max(ql - 2, 1), 60, kv // 2 + ql]
    res = _attend(q_lens, kv_lens, 2 * g, 2, d, 16, "bf16", window=window, seed=g + ql)
    _check_attend(res, d, kv_lens, True)


@pytest.mark.parametrize("dtype,max_q,q_lens", [("bf16", 1, [12, 1, 40]), ("bf16", 5, [200, 3, 64]), ("f32", 2, [90, 1, 33])])
def test_attention_more_units_than_the_host_expects(dtype, max_q, q_lens):
    """max_q_len and max_seq_len below the truth: the units that the host does not expect are
    done all the same, several a CTA."""
    N, Hq, Hkv, d, block = 36, 16, 4, 64, 16
    ql = [q_lens[n % 3] for n in range(N)]
    kv = [ql[n] + 11 * (n % 5) for n in range(N)]
    kc, vc, tables, keys, values = R.pages(kv, Hkv, d, block, DT[dtype], 5, DEV)
    g = torch.Generator().manual_seed(6)
    q = torch.randn(sum(ql), Hq, d, generator=g).to(DT[dtype]).to(DEV)
    cu = np.concatenate([[0], np.cumsum(ql)])
    out, lse = gdn.paged_attention(q, kc, vc, tables, _i32(kv), _i32(cu), max_q, max_seq_len=100, return_lse=True)
    gdn.gdn_check_status()
    res = []
    for n in range(N):
        sl = slice(cu[n], cu[n + 1])
        ref = R.attention(q[sl], keys[n], values[n], kv[n] - ql[n], d ** -0.5, 0)
        res.append((out[sl].double().cpu(), lse[sl].double().cpu(), ref))
    _check_attend(res, d, kv, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ql", [1, 24])
def test_attention_cut_and_whole_agree(ql, dtype):
    """The same requests with the sequences' bound given (units stay whole) and with a table of
    much more room (units are cut)."""
    N, Hq, Hkv, d, block = 5, 8, 2, 128, 16
    kv = [ql + x for x in (0, 37, 64, 90, 100)]
    kc, vc, tables, keys, values = R.pages(kv, Hkv, d, block, DT[dtype], 7, DEV)
    wide = torch.full((N, 4096), -1, dtype=torch.int32, device=DEV)
    wide[:, :tables.shape[1]] = tables
    g = torch.Generator().manual_seed(8)
    q = torch.randn(N * ql, Hq, d, generator=g).to(DT[dtype]).to(DEV)
    cu = _i32([n * ql for n in range(N + 1)])
    for table, bound in ((tables, 128), (wide, 0)):
        out, lse = gdn.paged_attention(q, kc, vc, table, _i32(kv), cu, ql, max_seq_len=bound, return_lse=True)
        gdn.gdn_check_status()
        res = []
        for n in range(N):
            sl = slice(n * ql, (n + 1) * ql)
            ref = R.attention(q[sl], keys[n], values[n], kv[n] - ql, d ** -0.5, 0)
            res.append((out[sl].double().cpu(), lse[sl].double().cpu(), ref))
        _check_attend(res, d, kv, dtype == "bf16")


def test_binding_refusals_and_the_librarys():
    """What does not fit is refused by name before the call, as ValueError (TypeError for dtypes
    and argument types); what the library refuses is a GdnError with its status and message."""
    bf = dict(dtype=torch.bfloat16, device=DEV)
    q, kc = torch.zeros(6, 4, 64, **bf), torch.zeros(8, 16, 2, 64, **bf)
    tables, sl, cu = torch.zeros(2, 4, dtype=torch.int32, device=DEV), _i32([3, 3]), _i32([0, 3, 6])

    def attend(**over):
        a = dict(q=q, k_cache=kc, v_cache=kc, block_tables=tables, seq_lens=sl, cu_seqlens=cu, max_q_len=3)
        a.update(over)
        return gdn.paged_attention(**a)

    for over, word in [(dict(q=q[:, :, ::2]), "q must be"), (dict(q=q[0]), "q must be"), (dict(q=None), "q must be"),
                       (dict(k_cache=kc.float()), "k_cache must be"), (dict(v_cache=kc[:4]), "v_cache must be"),
                       (dict(v_cache=kc.cpu()), "v_cache must be"), (dict(block_tables=tables.long()), "block_tables"),
                       (dict(block_tables=tables.t()), "block_tables"), (dict(seq_lens=sl[:1]), "seq_lens must be"),
                       (dict(cu_seqlens=cu[:2]), "cu_seqlens must be"), (dict(cu_seqlens=cu.cpu()), "cu_seqlens"),
                       (dict(workspace=torch.zeros(8)), "workspace must be"), (dict(max_q_len=1 << 40), "max_q_len")]:
        with pytest.raises(ValueError, match=word):
            attend(**over)
    for over in (dict(q=q.half()), dict(max_q_len="3"), dict(scale="a")):
        with pytest.raises(TypeError):
            attend(**over)
    for over, word in [(dict(window=-1), "window"), (dict(scale=0.0), "scale"),
                       (dict(q=q[:, :3].contiguous()), "Hq must be"),
                       (dict(workspace=torch.zeros(8, dtype=torch.uint8, device=DEV)), "workspace holds")]:
        with pytest.raises(gdn.GdnError, match=word) as e:
            attend(**over)
        assert e.value.status == gdn.GDN_EINVAL
    with pytest.raises(ValueError, match="out must be"):
        gdn.gdn_paged_attention(q, kc, kc, tables, sl, cu, q.float(), None, sl, 3)
    with pytest.raises(ValueError, match="lse must be"):
        gdn.gdn_paged_attention(q, kc, kc, tables, sl, cu, torch.empty_like(q), q, sl, 3)
    with pytest.raises(ValueError, match="out must be"):
        gdn.gdn_paged_attention(q, kc, kc, tables, sl, cu, None, None, sl, 3)
    with pytest.raises(ValueError, match="slot_map must be"):
        gdn.paged_write(q[:, :2], q[:, :2], cu, kc, kc.clone())
    with pytest.raises(ValueError, match="k and v must be"):
        gdn.paged_write(q, q, torch.zeros(6, dtype=torch.int32, device=DEV), kc, kc.clone())
    with pytest.raises(gdn.GdnError, match="block_size"):
        gdn.paged_plan(sl, sl, tables, cu, _i32([0, 3]), 12, 6)
    with pytest.raises(ValueError, match="num_tokens"):
        gdn.paged_plan(sl, sl, tables, cu, _i32([0, 3]), 16, -1)
    with pytest.raises(ValueError, match="ring_in must be"):
        gdn.paged_plan(sl, sl, tables, cu, cu, 16, 6)
    gate, pool = torch.zeros(6, 2, device=DEV), torch.zeros(4, 2, 64, 64, device=DEV)
    with pytest.raises(ValueError, match="state_pool must be"):
        gdn.recurrent_step(q[:, :2], q[:, :2], q[:, 2:], gate, gate, pool.bfloat16(), sl, cu)
    with pytest.raises(ValueError, match="log_alpha must be"):
        gdn.recurrent_step(q[:, :2], q[:, :2], q[:, 2:], gate[:5], gate, pool, sl, cu)
    with pytest.raises(gdn.GdnError, match="multiple of Hk"):
        gdn.recurrent_step(q, q, q[:, 2:], gate, gate, pool, sl, cu)
    assert torch.isfinite(attend()).all()


def test_binding_returns_ordinary_tensors():
    """Outputs can take part in autograd and in-place work like any other tensor, and inputs that
    require gradients are read as they are."""
    q = torch.randn(3, 4, 64, device=DEV, requires_grad=True)
    kc = torch.randn(4, 16, 2, 64, device=DEV)
    tables, sl, cu = _i32([[0]]), _i32([3]), _i32([0, 3])
    out, lse = gdn.paged_attention(q, kc, kc, tables, sl, cu, 3, return_lse=True)
    assert not out.requires_grad and out.is_contiguous() and lse.shape == (3, 4)
    w = torch.ones(64, device=DEV, requires_grad=True)
    (out * w).sum().backward()
    assert torch.allclose(w.grad, out.sum((0, 1)))
    p = gdn.paged_plan(_i32([0, 5]), _i32([2, 1]), torch.full((2, 4), -1, dtype=torch.int32, device=DEV),
                       torch.arange(8, dtype=torch.int32, device=DEV), _i32([0, 8]), 8, 3)
    assert [tuple(x.shape) for x in p] == [(3,), (2,), (3,), (3,), (2,), (2,)]
    kept = p.slot_map.clone()
    p.positions.fill_(-7)
    assert torch.equal(p.slot_map, kept) and p.cu_seqlens.tolist() == [0, 2, 3] and p.granted.tolist() == [1, 1]
