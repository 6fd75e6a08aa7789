"""The serving operators together, as examples/hybrid_serving.py runs them: what a request gets
must not depend on how its prompt is cut, who shares the batch, whose rows and blocks it takes
over, or how often it has to wait for blocks."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_gated_deltanet_gb300 import build
    build.build()


def _serve(cfg, requests, chunk, new=6):
    import hybrid_serving as hs
    server = hs.Server(hs.HybridStack(cfg, seed=3), chunk)
    for name, prompt in requests:
        server.submit(name, prompt, new)
    done, steps = {}, 0
    while server.running():
        for r in server.step():
            done[r["name"]] = r["out"]
        steps += 1
        assert steps < 500
    assert sorted(done) == sorted(n for n, _ in requests)
    # every block is free again
    head, count = server.stack.ring_state.tolist()
    free = [int(server.stack.ring[(head + i) % cfg.num_blocks]) for i in range(count)]
    assert sorted(free) == list(range(cfg.num_blocks))
    return done, server.last_logits


@pytest.mark.parametrize("window,num_blocks", [(0, 24), (40, 24), (0, 17)])
def test_requests_do_not_depend_on_the_batch(window, num_blocks):
    """fp32 stack: logits agree to the fp32 operators' accuracy through the layers."""
    import hybrid_serving as hs
    g = torch.Generator().manual_seed(0)
    requests = [(i, torch.randint(1000, (n,), generator=g).tolist()) for i, n in enumerate([1, 17, 63, 64, 130, 5, 40])]
    base = dict(layers="dada", hidden=128, delta_heads=4, delta_key_heads=2, delta_dim=32, heads=4, kv_heads=2,
                head_dim=32, dtype=torch.float32, window=window)
    alone = {}
    for r in requests:
        out, logits = _serve(hs.Config(rows=1, **base), [r], chunk=1000)
        alone[r[0]] = (out[r[0]], logits[r[0]])
    # few rows, few blocks (requests wait), pages of 8, prompts in pieces of 7
    out, logits = _serve(hs.Config(rows=3, block=8, num_blocks=num_blocks, **base), requests, chunk=7)
    for name, (want, want_logits) in alone.items():
        assert out[name] == want, name
        assert (logits[name] - want_logits).abs().max() < 2e-3 * want_logits.abs().max()


def test_bf16_stack_runs_and_agrees_roughly():
    """bf16, heads of 64 and 128 (the tensor-core kernels): logits of the last token."""
    import hybrid_serving as hs
    g = torch.Generator().manual_seed(1)
    requests = [(i, torch.randint(1000, (n,), generator=g).tolist()) for i, n in enumerate([200, 31, 90])]
    base = dict(layers="da", hidden=256, delta_heads=4, delta_key_heads=2, delta_dim=128, heads=8, kv_heads=2,
                head_dim=128)
    _, a = _serve(hs.Config(rows=3, **base), requests, chunk=1000, new=1)
    _, b = _serve(hs.Config(rows=2, **base), requests, chunk=50, new=1)
    for name in a:
        # two layers of bf16 activations: a few units of 2^-8
        assert (a[name] - b[name]).abs().max() < 16 * 2.0 ** -8 * a[name].abs().max()


def test_a_step_can_be_captured_in_a_graph():
    """Lengths are device data: one graph of the four operators serves steps of other lengths."""
    import chunkwise_gated_deltanet_gb300 as gdn
    dev, N, T, bs = torch.device("cuda"), 4, 24, 8
    g = torch.Generator(device=dev).manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    q, k, v = r(T, 4, 64).bfloat16(), r(T, 2, 64).bfloat16(), r(T, 2, 64).bfloat16()
    dk, dvv = torch.nn.functional.normalize(r(T, 2, 64), dim=-1).bfloat16(), r(T, 2, 64).bfloat16()
    la, be = -r(T, 2).abs(), torch.sigmoid(r(T, 2))
    kc, vc = (torch.zeros(64, bs, 2, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    pool0 = r(N, 2, 64, 64)
    idx = torch.arange(N, dtype=torch.int32, device=dev)
    ctx, new = (torch.zeros(N, dtype=torch.int32, device=dev) for _ in range(2))

    def run(state, pool):
        tables, ring, ring_state = state
        p = gdn.paged_plan(ctx, new, tables, ring, ring_state, bs, T)
        gdn.paged_write(k, v, p.slot_map, kc, vc)
        o = gdn.paged_attention(q, kc, vc, tables, p.seq_lens, p.cu_seqlens, T)
        y = gdn.recurrent_step(dk, dk, dvv, la, be, pool, idx, p.cu_seqlens, context_lens=ctx)
        return p, o, y

    def fresh():
        return (torch.full((N, 8), -1, dtype=torch.int32, device=dev), torch.arange(64, dtype=torch.int32, device=dev),
                torch.tensor([0, 64], dtype=torch.int32, device=dev))

    state, pool = fresh(), pool0.clone()
    new.copy_(torch.tensor([1, 2, 3, 4], dtype=torch.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(state, pool)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            captured = run(state, pool)
    torch.cuda.current_stream().wait_stream(side)
    for lens in ([1, 1, 1, 1], [20, 0, 3, 1], [0, 0, 0, 24], [7, 5, 11, 1]):
        new.copy_(torch.tensor(lens, dtype=torch.int32))
        for t, f in zip(state, fresh()):
            t.copy_(f)
        pool.copy_(pool0)
        graph.replay()
        torch.cuda.synchronize()
        got = [captured[0].seq_lens.clone(), captured[1][:sum(lens)].clone(), captured[2][:sum(lens)].clone(), pool.clone()]
        pool2 = pool0.clone()
        p, o, y = run(fresh(), pool2)
        want = [p.seq_lens, o[:sum(lens)], y[:sum(lens)], pool2]
        for a, b in zip(got, want):
            assert torch.equal(a, b), lens
    gdn.gdn_check_status()
