"""One decode block of the projections' model sizes, served: prompts in chunks, a fork, decode steps,
a compaction of the cache.

    python examples/decode_block.py [--w4]

Per step and block: the norm before, qkv_gate, the new keys and values into the paged cache,
attention over it with the gate, o, and the norms between this block and the router in one pass.
8 query heads on one key head of 128 elements, hidden width 8192, residual stream in FP32. Weights
and inputs are random. --w4 runs qkv_gate and o with 4-bit weights. Needs the built library and a GPU.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gemv_decode_projections_amd import binding, block  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 8192, 8, 1, 128, 16
ALPHA, EPS = 0.5, 1e-6


def four_bits(weight, group=128):
    """Group-scaled 4-bit form of a weight matrix: (packed nibbles, scales); offset 8."""
    n, k = weight.shape
    w = weight.float().view(n, k // group, group)
    scale = (w.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16)
    q = (torch.round(w / scale.float()).clamp(-8, 7) + 8).to(torch.uint8).view(n, k // 2, 2)
    return (q[..., 0] | q[..., 1] << 4).contiguous(), scale.view(n, k // group).contiguous()


class Block:
    """Weights of the block and what a serving program keeps for it."""

    def __init__(self, w4, gen):
        def weight(layer, dtype=torch.bfloat16):
            n, k, _, _ = binding.proj_layer_dims(layer)
            return (torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5).to(dtype)

        def scale():
            return (1 + 0.1 * torch.randn(HIDDEN, generator=gen, device="cuda")).to(torch.bfloat16)

        self.w = {"qkv_gate": weight("qkv_gate"), "o": weight("o"), "router": weight("router", torch.float32)}
        self.pre, self.post, self.router_pre = scale(), scale(), scale()
        self.w4 = {name: block.w4_prepare(*four_bits(self.w[name])) for name in ("qkv_gate", "o")} if w4 else {}
        for name in self.w:
            if name not in self.w4:
                binding.proj_prepare(name, self.w[name])
        self.ws = block.AttnWorkspace(DIM)

    def linear(self, name, x):
        if name not in self.w4:
            return binding.linear(name, x)
        out = torch.empty((x.shape[0], self.w4[name].n), dtype=x.dtype, device=x.device)
        block.w4_run(self.w4[name], x, out)
        return out

    def step(self, hidden, cache, table, q_start, kv_len, max_new):
        """The residual stream (FP32, tokens x HIDDEN) is updated in place; returns the router's logits."""
        tokens = hidden.shape[0]
        x = torch.empty((tokens, HIDDEN), dtype=torch.bfloat16, device=hidden.device)
        block.norm_run(None, hidden, x, weight_pre=self.pre, eps=EPS)
        q, k, v, gate = self.linear("qkv_gate", x).split([HEADS * DIM, DIM, DIM, HEADS * DIM], 1)
        block.kv_append(k.view(tokens, KV_HEADS, DIM), v.view(tokens, KV_HEADS, DIM), cache, table, q_start, kv_len)
        mixed = torch.empty((tokens, HEADS, DIM), dtype=torch.bfloat16, device=hidden.device)
        block.attn_run(q.view(tokens, HEADS, DIM), cache, table, q_start, kv_len, mixed, self.ws, max_q=max_new,
                       gate=gate.view(tokens, HEADS, DIM))
        o = self.linear("o", mixed.view(tokens, HEADS * DIM))
        block.norm_run(o, hidden, x, weight_pre=self.router_pre, weight_post=self.post, alpha=ALPHA, eps=EPS)
        return binding.linear("router", x)

    def release(self):
        for name in self.w:
            binding.proj_release(name)


class Server:
    """Sequences of one block: page lists, lengths, and the step's tables from them."""

    def __init__(self, model, n_pages):
        self.model, self.pool = model, block.PagePool(n_pages)
        self.cache = block.KvCache.empty(n_pages, PAGE, KV_HEADS, DIM)
        self.pages, self.length = {}, {}

    def add(self, name):
        self.pages[name], self.length[name] = [], 0

    def fork(self, name, new):
        self.pages[new], self.length[new] = self.pool.fork(self.pages[name]), self.length[name]

    def drop(self, name):
        self.pool.free(self.pages.pop(name))
        del self.length[name]

    def compact(self):
        src, dst = self.pool.compact()
        block.kv_copy_pages(self.cache, src, dst)
        self.pages = {name: self.pool.remap(p, src, dst) for name, p in self.pages.items()}
        return len(src)

    def step(self, inputs):
        """inputs: name -> residual rows (new tokens x HIDDEN, FP32). Returns name -> router logits."""
        copies = []
        for name, rows in inputs.items():
            pages, have = self.pages[name], self.length[name]
            if have % PAGE:                # the last page is written to: it has to be this sequence's own
                move = self.pool.writable(pages, len(pages) - 1)
                copies += [move] if move else []
            self.length[name] = have + rows.shape[0]
            pages += self.pool.alloc(-(-self.length[name] // PAGE) - len(pages))
        block.kv_copy_pages(self.cache, [c[0] for c in copies], [c[1] for c in copies])
        names = list(inputs)
        counts = [inputs[n].shape[0] for n in names]
        width = max(len(self.pages[n]) for n in names)
        device = self.cache.device
        table = torch.tensor([self.pages[n] + [-1] * (width - len(self.pages[n])) for n in names], dtype=torch.int32, device=device)
        starts = [sum(counts[:i]) for i in range(len(counts) + 1)]
        hidden = torch.cat([inputs[n] for n in names])
        logits = self.model.step(hidden, self.cache, table, torch.tensor(starts, dtype=torch.int32, device=device),
                                 torch.tensor([self.length[n] for n in names], dtype=torch.int32, device=device), max(counts))
        return dict(zip(names, logits.split(counts)))


def main(w4=False, prompts=(300, 45, 1), steps=20, seed=0):
    """Returns the last step's logits by sequence, and every input in order by sequence."""
    gen = torch.Generator("cuda").manual_seed(seed)
    server = Server(Block(w4, gen), 256)
    fed = {}

    def rows(n):
        return torch.randn(n, HIDDEN, generator=gen, device="cuda")

    def step(inputs):
        for name, x in inputs.items():
            fed[name] = torch.cat([fed[name], x]) if name in fed else x.clone()
        return server.step({name: x.clone() for name, x in inputs.items()})

    for i, n in enumerate(prompts):
        server.add("s%d" % i)
    while any(len(fed.get("s%d" % i, [])) < n for i, n in enumerate(prompts)):      # prompts in chunks of 128
        step({"s%d" % i: rows(min(128, n - len(fed.get("s%d" % i, [])))) for i, n in enumerate(prompts)
              if len(fed.get("s%d" % i, [])) < n})
    server.fork("s0", "fork")
    fed["fork"] = fed["s0"].clone()
    began = time.perf_counter()
    for i in range(steps):
        if i == steps // 2:                # one sequence ends, the cache closes up
            server.drop("s1")
            moved = server.compact()
        out = step({name: rows(1) for name in server.pages})
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    print("%d decode steps of %d to %d sequences, %s weights: %.0f us a step; %d pages moved, %d free"
          % (steps, len(prompts) + 1, len(server.pages), "4-bit" if w4 else "BF16", took / steps * 1e6, moved, server.pool.free_pages))
    model = server.model
    return out, fed, model


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--w4", action="store_true", help="qkv_gate and o with 4-bit weights")
    main(ap.parse_args().w4)[2].release()
