"""Host-side checks of the serving operators (CPU only: nothing is launched): every argument
that include/gdn.h rules out is refused with a message before any launch."""
import ctypes
import os

import pytest
import torch

import chunkwise_gated_deltanet_gb300 as gdn
from chunkwise_gated_deltanet_gb300 import build as gdn_build

A = [4096 * (i + 1) for i in range(16)]  # aligned addresses, never read


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.load_library()


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


def _plan(lib, **over):
    a = dict(ctx=A[0], new=A[1], bt=A[2], ring=A[3], rin=A[4], rout=A[5], cu=A[6], sl=A[7], sm=A[8], pos=A[9],
             gr=A[10], N=4, T=9, M=5, nb=40, bs=16)
    a.update(over)
    return lib.gdn_paged_plan(*(_p(a[x]) for x in ("ctx", "new", "bt", "ring", "rin", "rout", "cu", "sl", "sm",
                                                   "pos", "gr")), a["N"], a["T"], a["M"], a["nb"], a["bs"], None)


def _write(lib, **over):
    a = dict(k=A[0], v=A[1], sm=A[2], kc=A[3], vc=A[4], T=9, H=2, d=64, nb=40, bs=16, ks=128, vs=128, dt=1)
    a.update(over)
    return lib.gdn_paged_write(*(_p(a[x]) for x in ("k", "v", "sm", "kc", "vc")), a["T"], a["H"], a["d"], a["nb"],
                               a["bs"], a["ks"], a["vs"], a["dt"], None)


def _attend(lib, **over):
    a = dict(q=A[0], kc=A[1], vc=A[2], bt=A[3], sl=A[4], cu=A[5], out=A[6], lse=A[7], ws=A[8], wb=1 << 40, N=3,
             T=9, Hq=8, Hkv=2, d=64, M=5, nb=40, bs=16, mq=4, ms=0, w=0, scale=0.125, qs=512, dt=1)
    a.update(over)
    return lib.gdn_paged_attention(*(_p(a[x]) for x in ("q", "kc", "vc", "bt", "sl", "cu", "out", "lse", "ws")),
                                   *(a[x] for x in ("wb", "N", "T", "Hq", "Hkv", "d", "M", "nb", "bs", "mq", "ms",
                                                    "w", "scale", "qs", "dt")), None)


def _step(lib, **over):
    a = dict(q=A[0], k=A[1], v=A[2], la=A[3], be=A[4], sp=A[5], si=A[6], cu=A[7], cl=A[8], out=A[9], N=3, T=9,
             Hk=2, H=4, dk=64, dv=64, slots=7, qs=128, ks=128, vs=256, dt=1)
    a.update(over)
    return lib.gdn_recurrent_step(*(_p(a[x]) for x in ("q", "k", "v", "la", "be", "sp", "si", "cu", "cl", "out")),
                                  *(a[x] for x in ("N", "T", "Hk", "H", "dk", "dv", "slots", "qs", "ks", "vs",
                                                   "dt")), None)


@pytest.mark.parametrize("call,over,code,word", [
    (_plan, dict(N=-1), 1, "N, T"), (_plan, dict(T=-1), 1, "N, T"), (_plan, dict(M=0), 1, "max_blocks"),
    (_plan, dict(nb=0), 1, "num_blocks"), (_plan, dict(bs=12), 1, "block_size"), (_plan, dict(bs=0), 1, "block_size"),
    (_plan, dict(bs=2048), 1, "block_size"), (_plan, dict(nb=1 << 30), 1, "2^31"), (_plan, dict(M=1 << 30), 1, "2^31"),
    (_plan, dict(N=1 << 20, M=1 << 12), 1, "2^31"), (_plan, dict(ring=None), 1, "free_ring"),
    (_plan, dict(ctx=None), 1, "context_lens"), (_plan, dict(sm=None), 1, "slot_map"),
    (_plan, dict(cu=A[0] + 2), 1, "cu_seqlens is not 4-byte"), (_plan, dict(rout=A[4]), 1, "ring_out"),
    (_write, dict(dt=5), 2, "kv_dtype"), (_write, dict(T=-1), 1, "T >= 0"), (_write, dict(H=0), 1, "Hkv"),
    (_write, dict(d=48), 1, "d 16"), (_write, dict(bs=4), 1, "block_size"), (_write, dict(k=None), 1, "k must"),
    (_write, dict(vc=A[4] + 8), 1, "v_cache is not 16-byte"), (_write, dict(ks=64), 1, "k_stride"),
    (_write, dict(vs=132), 1, "v_stride"), (_write, dict(sm=A[2] + 1), 1, "slot_map"),
    (_attend, dict(dt=-1), 2, "qkv_dtype"), (_attend, dict(N=-1), 1, "N, T"), (_attend, dict(Hq=7), 1, "Hq"),
    (_attend, dict(Hkv=0), 1, "Hq"), (_attend, dict(d=96), 1, "d must"), (_attend, dict(bs=20), 1, "block_size"),
    (_attend, dict(M=0), 1, "max_blocks"), (_attend, dict(mq=-1), 1, "max_q_len"), (_attend, dict(w=-1), 1, "window"),
    (_attend, dict(ms=-4), 1, "max_seq_len"), (_attend, dict(scale=0.0), 1, "scale"),
    (_attend, dict(scale=float("nan")), 1, "scale"), (_attend, dict(scale=float("inf")), 1, "scale"),
    (_attend, dict(T=1 << 30), 1, "too large"), (_attend, dict(q=None), 1, "q must"),
    (_attend, dict(out=A[6] + 8), 1, "out is not"), (_attend, dict(bt=None), 1, "block_tables"),
    (_attend, dict(lse=A[7] + 2), 1, "lse"), (_attend, dict(qs=508), 1, "q_stride"),
    (_attend, dict(qs=516), 1, "q_stride"), (_attend, dict(ws=None), 1, "workspace"),
    (_attend, dict(wb=64), 1, "workspace holds 64"),
    (_attend, dict(M=(1 << 21) - 2, bs=1024, T=1 << 27, mq=1 << 27), 1, "max_seq_len"),
    (_attend, dict(M=(1 << 21) - 2, bs=1024, T=1 << 27, mq=1 << 27, d=32, qs=256, dt=0), 1, "max_seq_len"),
    (_step, dict(dt=3), 2, "qkv_dtype"), (_step, dict(N=-1), 1, "N, T"), (_step, dict(slots=0), 1, "slots"),
    (_step, dict(H=3), 1, "multiple of Hk"), (_step, dict(dk=48), 1, "dk and dv"), (_step, dict(dv=256), 1, "dk and dv"),
    (_step, dict(sp=None), 1, "state_pool"), (_step, dict(sp=A[5] + 4), 1, "16-byte"), (_step, dict(la=None), 1, "log_alpha"),
    (_step, dict(cl=A[8] + 3), 1, "context_lens"), (_step, dict(qs=120), 1, "q_stride"), (_step, dict(vs=260), 1, "v_stride"),
])
def test_invalid_arguments_are_refused(lib, call, over, code, word):
    assert call(lib, **over) == code
    assert word in lib.gdn_last_error().decode(), lib.gdn_last_error()


def test_nothing_to_do_is_no_error(lib):
    assert _write(lib, T=0, k=None, v=None, sm=None, kc=None, vc=None) == 0
    assert _attend(lib, T=0, q=None, out=None) == 0 and _attend(lib, N=0, bt=None) == 0
    assert _step(lib, T=0, q=None, out=None) == 0 and _step(lib, N=0, si=None) == 0


def test_workspace_query(lib):
    f = gdn.gdn_paged_attention_workspace_bytes
    assert f(8, 2, 64, 1, torch.bfloat16) > 0
    assert f(8, 3, 64, 1, torch.bfloat16) == 0 and f(8, 2, 65, 1, torch.float32) == 0
    assert f(8, 2, 64, -1, torch.float32) == 0


def test_binding_refuses_host_tensors_shapes_and_types(lib):
    i = torch.zeros(3, dtype=torch.int32)
    x = torch.zeros(4, 2, 16)
    cache = torch.zeros(3, 8, 2, 16)
    with pytest.raises(ValueError):
        gdn.gdn_paged_plan(i, i, i.view(3, 1), i, i[:2], i[1:], i, i, i, i, i, 8)
    with pytest.raises(ValueError):
        gdn.paged_write(x, x, i, cache, cache)
    with pytest.raises(TypeError):
        gdn.paged_write(x.half(), x.half(), i, cache.half(), cache.half())
    with pytest.raises(ValueError):
        gdn.gdn_paged_attention(x, cache, cache, i.view(3, 1), i, i, x, None, i, 1)
    with pytest.raises(ValueError):
        gdn.gdn_recurrent_step(x, x, x, x, x, x, i, i, x)


def test_serving_binding_computes_nothing():
    src = open(os.path.join(os.path.dirname(gdn.__file__), "serving.py")).read()
    for word in ("cumsum", "softmax", "index_copy", "scatter", "einsum", "matmul"):
        assert word not in src


def test_compiled_calls_check_their_arguments(lib):
    """The compiled binding itself: counts and types of arguments, and its own binding."""
    from chunkwise_gated_deltanet_gb300 import serving
    calls = serving._calls()
    for name, n in (("plan", 9), ("write", 6), ("attention", 14), ("step", 11), ("bind", 7)):
        for k in (0, 1, n - 1, n + 1):
            with pytest.raises(TypeError):
                getattr(calls, name)(*[None] * k)
        with pytest.raises((TypeError, ValueError)):
            getattr(calls, name)(*[None] * n)
        with pytest.raises((TypeError, ValueError)):
            getattr(calls, name)(*[3] * n) if name != "bind" else calls.bind(*[0] * n)
    with pytest.raises(ValueError, match="context_lens must be a CUDA tensor"):
        i = torch.zeros(3, dtype=torch.int32)
        gdn.paged_plan(i, i, i.view(3, 1), i, i[:2], 8, 3)
    with pytest.raises(ValueError, match="q must be a CUDA tensor, got list"):
        gdn.paged_attention([1], None, None, None, None, None, 1)
