"""A small hybrid stack on the library: delta-rule layers next to softmax attention.

    python -m kimi_delta_attention_prefill_gb300.hybrid            # serve a few ragged prompts

Every ``period``-th layer is softmax attention over a paged key/value cache (e4m3 by default),
the others are delta-rule layers whose whole memory is a 128 x 128 state a head.  The dense
projections around them are plain torch products with random weights: the point is how the
library's calls go together when a batch is served.

    prompt in chunks   delta layers: prefill from the running states;
                       attention: kv_append of the chunk's keys and values, attn_prefill_paged
    token by token     delta layers: decode; attention: kv_append, attn_decode_paged
"""
from __future__ import annotations

import torch

import kimi_delta_attention_prefill_gb300 as kda

D = kda.HEAD_DIM


class Pages:
    """Pages of one attention layer's cache (the page table, on the device, is the stack's)."""

    def __init__(self, n_pages, n_kv_heads, page_size, fp8, device):
        shape = (n_pages, n_kv_heads, page_size, D)
        kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
        raw = torch.uint8 if fp8 else torch.bfloat16
        self.k, self.v = (torch.zeros(shape, dtype=raw, device=device).view(kind) for _ in range(2))
        self.scales = {}
        if fp8:
            self.scales = {n: torch.full(shape[:3], 127, dtype=torch.uint8, device=device) for n in ("k_scale", "v_scale")}


class HybridStack:
    def __init__(self, n_layers=4, period=4, heads=8, kv_heads=2, width=512, n_seq=3, max_tokens=2048, page_size=64,
                 fp8=True, window=0, n_sink=0, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.heads, self.kv_heads, self.width, self.n_seq = heads, kv_heads, width, n_seq
        self.window, self.n_sink, self.page_size, self.device = window, n_sink, page_size, device
        self.max_pages = (max_tokens + page_size - 1) // page_size
        n_pages = n_seq * self.max_pages
        # one page table serves every attention layer: the pages of a sequence, handed out in any order
        self.table = torch.randperm(n_pages, generator=g, device=device).to(torch.int32).view(n_seq, self.max_pages)
        self.length = torch.zeros(n_seq, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        w = lambda *s: torch.randn(s, generator=g, device=device, dtype=torch.float32).mul_(s[0] ** -0.5).to(torch.bfloat16)
        self.layers = []
        for i in range(n_layers):
            if i % period == period - 1:
                self.layers.append(dict(kind="attention", qkv=w(width, (heads + 2 * kv_heads) * D), out=w(heads * D, width),
                                        pages=Pages(n_pages, kv_heads, page_size, fp8, device)))
            else:
                self.layers.append(dict(kind="delta", qkv=w(width, 3 * heads * D), gate=w(width, heads * D), beta=w(width, heads),
                                        out=w(heads * D, width),
                                        state=torch.zeros(n_seq, heads, D, D, dtype=torch.float32, device=device)))

    def _delta_inputs(self, layer, x):
        q, k, v = (x @ layer["qkv"]).view(-1, 3, self.heads, D).unbind(1)
        unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).to(torch.bfloat16)
        g = -5.0 * torch.sigmoid((x @ layer["gate"]).float().view(-1, self.heads, D) - 4.0)
        beta = torch.sigmoid((x @ layer["beta"]).float())
        return unit(q), unit(k), v.contiguous(), g, beta

    def _step(self, x, cu, n_tok):
        """x [T, width] bf16, packed by cu; n_tok: every sequence's tokens (decode), or None (prefill)."""
        new = cu.diff()
        kv_len = self.length + new
        for layer in self.layers:
            h = torch.nn.functional.rms_norm(x.float(), (self.width,)).to(torch.bfloat16)
            if layer["kind"] == "delta":
                args = self._delta_inputs(layer, h)
                if n_tok is None:
                    o, layer["state"], _ = kda.prefill(*args, cu, S_in=layer["state"], dev_status=self.status)
                else:
                    o = kda.decode(*(t.view(self.n_seq, n_tok, *t.shape[1:]) for t in args), layer["state"],
                                   dev_status=self.status).to(torch.bfloat16)
            else:
                qkv = (h @ layer["qkv"]).view(-1, self.heads + 2 * self.kv_heads, D)  # its rows are used where they lie
                q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
                p = layer["pages"]
                kda.kv_append(k, v, p.k, p.v, self.table, cu, self.length, **p.scales, dev_status=self.status)
                seen = dict(window=self.window, n_sink=self.n_sink, dev_status=self.status, **p.scales)
                if n_tok is None:
                    o = kda.attn_prefill_paged(q, p.k, p.v, self.table, cu, kv_len, **seen)
                else:
                    o = kda.attn_decode_paged(q.view(self.n_seq, n_tok, self.heads, D), p.k, p.v, self.table, kv_len, **seen)
            x = x + o.reshape(-1, self.heads * D) @ layer["out"]
        self.length = kv_len
        return x

    def prompt(self, x, cu_seqlens):
        """The next chunk of every sequence's prompt: x [T, width] bf16, cu_seqlens [n_seq + 1] int32."""
        return self._step(x, cu_seqlens, None)

    def decode(self, x):
        """The next tokens: x [n_seq, n_tok, width] bf16, n_tok <= 4."""
        n, n_tok, _ = x.shape
        cu = torch.arange(0, n * n_tok + 1, n_tok, dtype=torch.int32, device=x.device)
        return self._step(x.reshape(-1, self.width), cu, n_tok).view_as(x)


def main():
    prompts = [300, 77, 1]
    stack = HybridStack(n_seq=len(prompts), max_tokens=1024)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    for part in range(2):  # the prompts in two chunks each
        new = [n - n // 2 if part == 0 else n // 2 for n in prompts]
        cu = torch.tensor([0] + new, dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)
        y = stack.prompt(rows(sum(new), stack.width), cu)
        print(f"chunk {part}: {new} tokens, |y| {float(y.float().abs().mean()):.4f}")
    for i in range(3):
        y = stack.decode(rows(len(prompts), 1, stack.width))
    print(f"3 tokens more: lengths {stack.length.tolist()}, |y| {float(y.float().abs().mean()):.4f}")
    if int(stack.status):
        raise SystemExit(f"library status {kda.status_string(int(stack.status))}")


if __name__ == "__main__":
    main()
