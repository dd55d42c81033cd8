"""A whole decoder layer on this library: attention over a paged 4-bit cache, then routed experts.

    python examples/decoder_layer.py            (needs the built library and a GB300)

Several sequences run at once.  A prompt enters in one piece (`prompt`): its keys and
values are appended to the cache, rotated on the way, and its queries attend causally
over the prompt.  A further piece of it (`chunk`) reads what is cached back and attends
over that and itself.  Tokens after it come one per sequence (`decode`), attending over
the 4-bit cache; that step has fixed shapes and no host work, so it is captured into a
CUDA graph once and replayed.  Projections are plain matrix products; the norms are a
line of torch each.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import router_softmax_top_gb300 as moe  # noqa: E402


def rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class DecoderLayer:
    def __init__(self, experts, layer, hidden, hq, hkv, head_dim, n_experts, *, seqs, longest, page_size=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, m):
            return (torch.randn(n, m, generator=g, device="cuda") * n ** -0.5).bfloat16()
        self.experts, self.layer = experts, layer
        self.hq, self.hkv, self.d, self.page_size = hq, hkv, head_dim, page_size
        self.w_qkv, self.w_o = weight(hidden, (hq + 2 * hkv) * head_dim), weight(hq * head_dim, hidden)
        self.w_router = weight(hidden, n_experts).float()
        width = -(-longest // page_size)
        self.pages = moe.kv_pages(seqs * width, hkv, head_dim, page_size)
        # every sequence has its pages from the start; a server hands them out as sequences grow
        self.table = torch.randperm(seqs * width, generator=g, device="cuda").to(torch.int32).view(seqs, width)
        self.cos, self.sin = moe.rope_table(longest, head_dim)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.one_each = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")

    def _append(self, x, cu):
        qkv = (rms(x).bfloat16() @ self.w_qkv).view(x.shape[0], self.hq + 2 * self.hkv, self.d)
        q, k, v = qkv.split([self.hq, self.hkv, self.hkv], 1)
        q, k = moe.kv_append(self.pages, self.table, self.lens, cu, k, v, page_size=self.page_size, q=q, cos=self.cos,
                             sin=self.sin, status=self.status)
        return q, k, v

    def _rest(self, x, attended):
        x = x + (attended.flatten(1) @ self.w_o).float()
        h = rms(x)
        # prompts go through the expert cache in the batches that it was made for
        most = self.experts.cfg.max_tokens
        y = torch.empty_like(h)
        for i in range(0, x.shape[0], most):
            part = h[i:i + most].contiguous()
            self.experts.forward(self.layer, part @ self.w_router, part, out=y[i:i + most])
        return x + y

    def prompt(self, x, cu):
        """x [tokens, hidden] fp32, sequence s's tokens [cu[s], cu[s+1]); nothing is cached before."""
        q, k, v = self._append(x, cu)
        out = self._rest(x, moe.prompt_attention(q, k, v, cu, status=self.status))
        self.lens += cu.diff()
        return out

    def chunk(self, x, cu, n_cached):
        """More of the prompts, after n_cached tokens (over all sequences) of which the cache knows."""
        q, _, _ = self._append(x, cu)
        new = cu.diff()
        # the pieces before, and this one, as the cache holds them
        cu_k = torch.cat([cu[:1], (self.lens + new).cumsum(0, dtype=torch.int32)])
        k, v = moe.kv_read(self.pages, self.table, torch.zeros_like(self.lens), cu_k, n_cached + x.shape[0],
                           page_size=self.page_size, n_kv_heads=self.hkv, head_dim=self.d, status=self.status)
        out = self._rest(x, moe.prompt_attention(q, k, v, cu, cu_k, status=self.status))
        self.lens += new
        return out

    def decode(self, x):
        """One token of every sequence."""
        q, _, _ = self._append(x, self.one_each)
        self.lens += 1
        return self._rest(x, moe.kv_attention(q, self.pages, self.table, self.lens, page_size=self.page_size,
                                              n_kv_heads=self.hkv, status=self.status))


def build(seqs=3, longest=512):
    import synth
    sh = synth.TINY
    store = torch.empty(sh.L * sh.E * synth.expert_bytes(sh.H, sh.F), dtype=torch.uint8, pin_memory=True)
    synth.fill_store(store.data_ptr(), sh.L, sh.E, sh.H, sh.F, 0)
    experts = moe.MoECache(n_layers=sh.L, n_experts=sh.E, top_k=sh.k, hidden=sh.H, ffn=sh.F, slots_per_layer=sh.E,
                           max_tokens=4, store=store, fill_mode=moe.MOE_FILL_PULL)
    return DecoderLayer(experts, 0, sh.H, 4, 2, 64, sh.E, seqs=seqs, longest=longest), sh.H


def main():
    layer, hidden = build()
    lens = [100, 37, 200]
    cu = torch.tensor([0, 100, 137, 337], dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lens), hidden, device="cuda")
    print("prompt", tuple(layer.prompt(x, cu).shape))
    more = torch.tensor([0, 5, 5, 25], dtype=torch.int32, device="cuda")
    print("chunk", tuple(layer.chunk(torch.randn(25, hidden, device="cuda"), more, sum(lens)).shape))
    step = torch.randn(3, hidden, device="cuda")
    layer.decode(step)                           # once outside the capture: set-up of the libraries
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.decode(step)
    for _ in range(16):
        graph.replay()                           # the graph moves lens on by itself
    torch.cuda.synchronize()
    assert layer.experts.sync() == moe.MOE_OK
    print("decode", tuple(out.shape), "lengths", layer.lens.tolist(), moe.status_message(layer.status) or "status ok")


if __name__ == "__main__":
    main()
