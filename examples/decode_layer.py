"""One attention layer of a serving loop: prompts enter, then tokens are decoded.

    python examples/decode_layer.py [--steps N] [--cache e4m3|fp16]

Each step runs, on one stream and without a copy to the host:

    plan       pages and slots for the tokens that enter
    QKV        a W8A16 product whose output is read in place as q, k and v
    append     the new keys and values into the paged cache
    attention  of one new token per request over its pages
    output     a W4A16 product

The decode step is captured into a graph once and replayed; the lengths that
change from step to step stay on the device.  The last line compares the
outputs with the same layer computed in fp64 over an ordinary, unpaged cache.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_quantized_gemm_qgemm_amd as qg  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 1024, 16, 4, 64, 16
QKV = (HEADS + 2 * KV_HEADS) * DIM


class Layer:
    """The weights, packed once, and the cache with its free pages."""

    def __init__(self, batch, max_len, cache, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(shape):
            return torch.randn(shape, generator=g, device=device)

        self.w_qkv = torch.randint(-127, 128, (HIDDEN, QKV), generator=g, device=device,
                                   dtype=torch.int8)
        self.s_qkv = (rand(QKV).abs() * 2e-4 + 5e-4).half()
        self.p_qkv = qg.qgemm_prepack("w8a16", self.w_qkv, HIDDEN, QKV)
        self.w_out = torch.randint(0, 256, (HEADS * DIM // 2, HIDDEN), generator=g, device=device,
                                   dtype=torch.uint8)
        self.s_out = (rand(HIDDEN).abs() * 2e-3 + 5e-3).half()
        self.p_out = qg.qgemm_prepack("w4a16", self.w_out, HEADS * DIM, HIDDEN)

        self.batch, self.max_len = batch, max_len
        width = -(-max_len // PAGE)
        self.pages = batch * width
        dtype = torch.float8_e4m3fn if cache == "e4m3" else torch.float16
        shape = (self.pages, 2, KV_HEADS, PAGE, DIM)
        pool = torch.zeros(shape, dtype=torch.uint8 if cache == "e4m3" else dtype, device=device)
        self.k_cache, self.v_cache = (pool[:, j].view(dtype) for j in (0, 1))
        self.scales = [torch.full((KV_HEADS,), 1 / 32, device=device) if cache == "e4m3" else None
                       for _ in range(2)]
        self.table = torch.full((batch, width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        # the free pages in an order of their own; `taken` of them are gone
        self.order = torch.randperm(self.pages, generator=g, device=device, dtype=torch.int32)
        self.free = self.order.clone()
        self.taken = torch.zeros(1, dtype=torch.int64, device=device)
        self.at = torch.arange(self.pages, device=device)
        self.workspace = torch.empty(max(16, qg.qgemm_paged_attention_workspace_bytes(
            batch, HEADS, KV_HEADS, DIM, max_len)), dtype=torch.uint8, device=device)

    def enter(self, x, added, plan_out):
        """Cache the tokens x [tokens, HIDDEN], added[b] of them for request b;
        returns their queries [tokens, HEADS, DIM]."""
        lens, _, cu_pages, slots = qg.qgemm_kv_plan(self.table, self.lens, added, self.free, PAGE,
                                                    x.shape[0], out=plan_out)
        qkv = qg.qgemm_w8a16(x, self.p_qkv, self.s_qkv, QKV)
        q, k, v = qkv.split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], dim=1)
        qg.qgemm_kv_append(k.unflatten(1, (KV_HEADS, DIM)), v.unflatten(1, (KV_HEADS, DIM)), slots,
                           self.k_cache, self.v_cache, *self.scales)
        self.lens.copy_(lens)
        self.taken.add_(cu_pages[-1:])
        self.free.copy_(self.order[(self.at + self.taken) % self.pages])
        return q.unflatten(1, (HEADS, DIM))

    def decode(self, x, added, plan_out):
        """One new token per request: x [batch, HIDDEN] -> [batch, HIDDEN]."""
        q = self.enter(x, added, plan_out)
        o = qg.qgemm_paged_attention(q, self.k_cache, self.v_cache, self.table, self.lens,
                                     *self.scales, max_len=self.max_len, workspace=self.workspace)
        return qg.qgemm_w4a16(o.flatten(1), self.p_out, self.s_out, HIDDEN)


def plan_buffers(batch, tokens, device):
    i32 = {"dtype": torch.int32, "device": device}
    return (torch.empty(batch, **i32), torch.empty(batch + 1, **i32), torch.empty(batch + 1, **i32),
            torch.empty(tokens, dtype=torch.int64, device=device))


def reference(layer, history):
    """The last token's output of each request in fp64; history[b] [n, HIDDEN]."""
    w_qkv = (layer.w_qkv.double() * layer.s_qkv.double()).cpu()
    codes = torch.stack([layer.w_out & 15, layer.w_out >> 4], dim=1).flatten(0, 1).double() - 8
    w_out = (codes * layer.s_out.double()).cpu()
    outs = []
    for x in history:
        qkv = (x.double().cpu() @ w_qkv).half()      # the product's own rounding
        q, k, v = qkv.split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], dim=1)
        k, v = (t.unflatten(1, (KV_HEADS, DIM)) for t in (k, v))
        if layer.scales[0] is not None:
            k, v = ((t.float() * 32).clamp(-448, 448).to(torch.float8_e4m3fn).double() / 32
                    for t in (k, v))
        k, v = (t.double().repeat_interleave(HEADS // KV_HEADS, dim=1) for t in (k, v))
        s = torch.einsum("hd,nhd->hn", q[-1].view(HEADS, DIM).double(), k) * DIM ** -0.5
        o = torch.einsum("hn,nhd->hd", torch.softmax(s, dim=1), v).half()
        outs.append(o.flatten().double() @ w_out)
    return torch.stack(outs)


def run(steps=40, cache="e4m3", prompts=(5, 130, 1, 64, 47), device="cuda", seed=1):
    """Returns (outputs of the last step, the same in fp64)."""
    batch, g = len(prompts), torch.Generator(device=device).manual_seed(seed)
    layer = Layer(batch, max(prompts) + steps, cache, device)
    tokens = sum(prompts)
    x = torch.randn((tokens, HIDDEN), generator=g, device=device).half()
    added = torch.tensor(prompts, dtype=torch.int32, device=device)
    layer.enter(x, added, plan_buffers(batch, tokens, device))
    history = [[part] for part in x.split(list(prompts))]

    x, added = torch.empty((batch, HIDDEN), dtype=torch.float16, device=device), torch.ones_like(added)
    buffers, graph, y = plan_buffers(batch, batch, device), None, None
    for step in range(steps):
        x.copy_(torch.randn((batch, HIDDEN), generator=g, device=device))
        for b in range(batch):
            history[b].append(x[b:b + 1].clone())
        if step == 1:      # the first step ran eagerly: capture one like it, then replay
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = layer.decode(x, added, buffers)
        if graph is None:
            y = layer.decode(x, added, buffers)
        else:
            graph.replay()
    torch.cuda.synchronize()
    assert layer.lens.tolist() == [n + steps for n in prompts]
    return y.double().cpu(), reference(layer, [torch.cat(h) for h in history])


def main():
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=40)
    parser.add_argument("--cache", choices=["e4m3", "fp16"], default="e4m3")
    args = parser.parse_args()
    y, ref = run(args.steps, args.cache)
    print(f"{args.steps} steps, {args.cache} cache: relative error "
          f"{float((y - ref).norm() / ref.norm()):.2e} against fp64")


if __name__ == "__main__":
    main()
