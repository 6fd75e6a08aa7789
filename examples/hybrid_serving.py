"""Continuous batching of a small hybrid stack: gated-delta layers beside attention layers.

Every request has a row.  A step packs the new tokens of all running requests (a chunk of the
prompt, or the token just sampled) and runs, for the whole batch,

    paged_plan        once: block tables, slots, positions and offsets from the lengths
    recurrent_step    in each gated-delta layer: states of a pool, by the request's row
    paged_write,
    paged_attention   in each attention layer: keys and values in pages

Requests end, their blocks are given back by the next plan, and waiting ones take their rows.
A request that gets no blocks is left out of the step (its state is passed over, its tokens
attend to nothing) and comes again in the next one; when none gets any, the last to come gives
its blocks back and starts over once another has ended.  Weights are random: the example shows the
calls, not a model.

    python examples/hybrid_serving.py --requests 40 --rows 16 --new-tokens 24
"""
from __future__ import annotations

import argparse
import dataclasses
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunkwise_gated_deltanet_gb300 as gdn  # noqa: E402


@dataclasses.dataclass
class Config:
    layers: str = "ddda"        # d: gated delta, a: attention
    hidden: int = 512
    vocab: int = 1000
    delta_heads: int = 8
    delta_key_heads: int = 4
    delta_dim: int = 64
    heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    window: int = 0
    dtype: torch.dtype = torch.bfloat16
    rows: int = 16              # requests running at a time
    block: int = 16
    num_blocks: int = 512
    max_len: int = 1024


def _rotate(x, positions):
    """Rotary position embedding of [T, heads, d]."""
    half = x.shape[-1] // 2
    freq = torch.exp(torch.arange(half, device=x.device) * (-9.21 / half))
    angle = positions[:, None, None] * freq
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1).to(x.dtype)


def _norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def _unit(x):
    return (x.float() * torch.rsqrt(x.float().square().sum(-1, keepdim=True) + 1e-6)).to(x.dtype)


class HybridStack:
    """Weights, caches and one step of the stack."""

    def __init__(self, cfg: Config, seed: int = 0):
        self.cfg, c, dev = cfg, cfg, torch.device("cuda")
        g = torch.Generator(device=dev).manual_seed(seed)

        def weight(n, m):
            return (torch.randn(n, m, generator=g, device=dev) / n ** 0.5).to(c.dtype)

        self.embed = weight(c.vocab, c.hidden) * c.vocab ** 0.5
        self.blocks = []
        for kind in c.layers:
            if kind == "d":
                wide = (2 * c.delta_key_heads + c.delta_heads) * c.delta_dim
                self.blocks.append(dict(inp=weight(c.hidden, wide), gates=weight(c.hidden, 2 * c.delta_heads),
                                        out=weight(c.delta_heads * c.delta_dim, c.hidden),
                                        pool=torch.zeros(c.rows, c.delta_heads, c.delta_dim, c.delta_dim, device=dev)))
            else:
                pages = (c.num_blocks, c.block, c.kv_heads, c.head_dim)
                self.blocks.append(dict(inp=weight(c.hidden, (c.heads + 2 * c.kv_heads) * c.head_dim),
                                        out=weight(c.heads * c.head_dim, c.hidden),
                                        k=torch.zeros(pages, dtype=c.dtype, device=dev),
                                        v=torch.zeros(pages, dtype=c.dtype, device=dev)))
        self.tables = torch.full((c.rows, -(-c.max_len // c.block)), -1, dtype=torch.int32, device=dev)
        self.ring = torch.arange(c.num_blocks, dtype=torch.int32, device=dev)
        self.ring_state = torch.tensor([0, c.num_blocks], dtype=torch.int32, device=dev)
        self.index = torch.arange(c.rows, dtype=torch.int32, device=dev)

    def step(self, tokens, context_lens, new_lens, max_new: int, max_len: int):
        """tokens [T], the running requests' new ones; context_lens, new_lens [rows] int32.
        Returns the logits after each request's last token [rows, vocab] and the plan."""
        c, T = self.cfg, tokens.numel()
        plan = gdn.paged_plan(context_lens, new_lens, self.tables, self.ring, self.ring_state, c.block, T)
        self.ring_state = plan.ring_state
        index = torch.where(plan.granted > 0, self.index, -1)
        x = self.embed[tokens]
        for kind, w in zip(c.layers, self.blocks):
            h = _norm(x)
            y = h @ w["inp"]
            if kind == "d":
                y = y.view(T, 2 * c.delta_key_heads + c.delta_heads, c.delta_dim)
                kh = c.delta_key_heads
                gates = (h @ w["gates"]).float()
                log_alpha = torch.nn.functional.logsigmoid(gates[:, :c.delta_heads] + 3).contiguous()
                beta = torch.sigmoid(gates[:, c.delta_heads:]).contiguous()
                # keys, queries and values are slices of one projection; v goes in as it is
                o = gdn.recurrent_step(_unit(y[:, :kh]), _unit(y[:, kh:2 * kh]), y[:, 2 * kh:], log_alpha, beta,
                                       w["pool"], index, plan.cu_seqlens, context_lens=context_lens)
            else:
                y = y.view(T, c.heads + 2 * c.kv_heads, c.head_dim)
                q = _rotate(y[:, :c.heads], plan.positions)
                k = _rotate(y[:, c.heads:c.heads + c.kv_heads], plan.positions)
                gdn.paged_write(k, y[:, c.heads + c.kv_heads:], plan.slot_map, w["k"], w["v"])
                o = gdn.paged_attention(q, w["k"], w["v"], self.tables, plan.seq_lens, plan.cu_seqlens, max_new,
                                        max_seq_len=max_len, window=c.window)
            x = x + o.flatten(1) @ w["out"]
        if T == 0:  # a step that only gives blocks back
            return torch.zeros(c.rows, c.vocab, device=x.device), plan
        last = (plan.cu_seqlens[1:].long() - 1).clamp(min=0)
        return (_norm(x[last]) @ self.embed.T).float(), plan


class Server:
    """Requests on the rows of a HybridStack; greedy sampling."""

    def __init__(self, stack: HybridStack, chunk: int = 64):
        self.stack, self.chunk = stack, chunk
        n = stack.cfg.rows
        self.todo, self.row, self.held, self.ended = [], [None] * n, [0] * n, [False] * n
        self.came, self.hold = [], False  # rows in the order of coming; no one comes in while on hold
        self.last_logits = {}

    def submit(self, name, prompt, new_tokens: int):
        self.todo.append(dict(name=name, prompt=list(prompt), out=[], want=new_tokens))

    def running(self) -> bool:
        return bool(self.todo) or any(r is not None for r in self.row) or any(self.ended)

    def step(self):
        """One step of the batch.  Returns the requests that ended."""
        n, new, tokens = len(self.row), [0] * len(self.row), []
        for i in range(n):
            if self.ended[i]:  # its blocks go back with this plan; the row is free in the next
                new[i] = -1
                continue
            if self.row[i] is None and self.todo and not self.hold:
                self.row[i], self.held[i] = self.todo.pop(0), 0
                self.came.append(i)
            r = self.row[i]
            if r is not None:
                part = (r["prompt"] + r["out"])[self.held[i]:][:self.chunk]
                new[i] = len(part)
                tokens += part
        dev = torch.device("cuda")
        lens = torch.tensor([self.held, new], dtype=torch.int32).to(dev, non_blocking=True)
        ids = torch.tensor(tokens, dtype=torch.int64).to(dev, non_blocking=True)
        logits, plan = self.stack.step(ids, lens[0], lens[1], max(new + [1]),
                                       max(h + max(x, 0) for h, x in zip(self.held, new)))
        best, granted = logits.argmax(-1).tolist(), plan.granted.tolist()
        done, freed = [], any(self.ended)
        for i in range(n):
            if self.ended[i]:
                self.ended[i], self.held[i] = False, 0
            r = self.row[i]
            if r is None or new[i] <= 0 or not granted[i]:
                continue
            self.held[i] += new[i]
            if self.held[i] == len(r["prompt"]) + len(r["out"]):
                r["out"].append(best[i])
                self.last_logits[r["name"]] = logits[i]
            if len(r["out"]) >= r["want"]:
                done.append(r)
                self._leave(i)
                self.hold = False
        if not (freed or any(x > 0 and ok for x, ok in zip(new, granted))):
            if len(self.came) < 2:
                raise RuntimeError("a request needs more blocks than there are")
            self.todo.insert(0, self.row[self.came[-1]])
            self._leave(self.came[-1])
            self.hold = True
        return done

    def _leave(self, i):
        self.row[i], self.ended[i] = None, True
        self.came.remove(i)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=40)
    ap.add_argument("--rows", type=int, default=16)
    ap.add_argument("--new-tokens", type=int, default=24)
    ap.add_argument("--chunk", type=int, default=64)
    a = ap.parse_args()
    cfg = Config(rows=a.rows, num_blocks=32 * a.rows)
    server = Server(HybridStack(cfg), a.chunk)
    g = torch.Generator().manual_seed(1)
    for i in range(a.requests):
        size = int(torch.randint(1, 300, (1,), generator=g))
        server.submit(i, torch.randint(cfg.vocab, (size,), generator=g).tolist(), a.new_tokens)
    server.step()  # loads libraries and kernels
    torch.cuda.synchronize()
    steps = made = 0
    began = time.perf_counter()
    while server.running():
        for r in server.step():
            made += len(r["out"])
        steps += 1
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    gdn.gdn_check_status()
    print(f"{a.requests} requests on {a.rows} rows: {made} tokens in {steps} steps, {took:.2f} s "
          f"({made / took:.0f} tokens/s, {1e3 * took / steps:.2f} ms a step)")


if __name__ == "__main__":
    main()
