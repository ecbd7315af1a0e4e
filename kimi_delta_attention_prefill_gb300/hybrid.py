"""A small hybrid stack on the library: delta-rule layers next to softmax attention.

    python -m kimi_delta_attention_prefill_gb300.hybrid            # serve a few ragged prompts

Every ``period``-th layer is softmax attention over a paged key/value cache (e4m3 by default),
the others are delta-rule layers whose whole memory is a 128 x 128 state a head.  ``kinds`` names
the layers one by one instead, and may hold "decay" layers: linear attention whose state decays by
one factor a head, with keys shared by several heads.  The dense projections around them are plain
torch products with random weights: the point is how the library's calls go together when a batch
is served.

    prompt in chunks   delta layers: prefill from the running states; decay layers: lin_prefill;
                       attention: kv_append of the chunk's keys and values, attn_prefill_paged
    token by token     delta layers: decode; decay layers: lin_decode (with n_commit where drafted
                       tokens are refused); attention: kv_append, attn_decode_paged
    between layers     x + f(N(x)), or with ``post_norm`` x + scale sigmoid(gate) N'(f(N(x))): one
                       block_norm a layer, over a residual stream in fp32
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
                 fp8=True, window=0, n_sink=0, seed=0, device="cuda", kinds=None, post_norm=False, block_scale=1.0):
        """kinds: "delta", "decay" or "attention" for each layer (None: by n_layers and period).  With post_norm every
        layer's output is normed, gated and scaled by block_scale before it joins the residual stream, and the
        stack returns its last norm's rows."""
        if kinds is None:
            kinds = ["attention" if i % period == period - 1 else "delta" for i in range(n_layers)]
        if any(kind not in ("delta", "decay", "attention") for kind in kinds):
            raise ValueError(f"a layer is delta, decay or attention, got {list(kinds)}")
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
        states = lambda: torch.zeros(n_seq, heads, D, D, dtype=torch.float32, device=device)
        for i, kind in enumerate(kinds):
            if kind == "attention":
                self.layers.append(dict(kind="attention", qkv=w(width, (heads + 2 * kv_heads) * D), out=w(heads * D, width),
                                        pages=Pages(n_pages, kv_heads, page_size, fp8, device)))
            elif kind == "decay":
                # memories from some tokens to thousands: of the first half of these layers fixed, then by token
                slopes = -torch.exp2(-8.0 * torch.arange(1, heads + 1, device=device, dtype=torch.float32) / heads)
                self.layers.append(dict(kind=kind, qkv=w(width, (heads + 2 * kv_heads) * D), gate=w(width, heads * D),
                                        decay=w(width, heads) if i >= len(kinds) / 2 else None, slopes=slopes,
                                        norm=torch.ones(D, device=device), out=w(heads * D, width), state=states()))
            else:
                self.layers.append(dict(kind="delta", qkv=w(width, 3 * heads * D), gate=w(width, heads * D), beta=w(width, heads),
                                        out=w(heads * D, width), state=states()))
        self.norms, self.block_scale = None, block_scale
        if post_norm:
            ones = lambda: torch.ones(width, device=device)
            self.norms = [dict(pre=ones(), post=ones(), gate=w(width, width)) for _ in kinds]
            self.last_norm = ones()

    def _delta_inputs(self, layer, x):
        q, k, v = (x @ layer["qkv"]).view(-1, 3, self.heads, D).unbind(1)
        unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).to(torch.bfloat16)
        g = -5.0 * torch.sigmoid((x @ layer["gate"]).float().view(-1, self.heads, D) - 4.0)
        beta = torch.sigmoid((x @ layer["beta"]).float())
        return unit(q), unit(k), v.contiguous(), g, beta

    def _decay_inputs(self, layer, x):
        q, k, v = (x @ layer["qkv"]).view(-1, self.heads + 2 * self.kv_heads, D).split([self.kv_heads, self.kv_heads, self.heads], 1)
        unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).to(torch.bfloat16)
        g = layer["slopes"]
        if layer["decay"] is not None:
            g = g * torch.nn.functional.softplus((x @ layer["decay"]).float())
        return (unit(q), unit(k), v, g), (x @ layer["gate"]).view(-1, self.heads, D)

    def _mix(self, layer, h, cu, kv_len, n_tok, n_commit):
        """The layer's mixing of tokens: h [T, width] bf16 -> [T, heads, 128] bf16."""
        by_seq = lambda t: t if t.dim() == 1 else t.view(self.n_seq, n_tok, *t.shape[1:])
        if layer["kind"] == "delta":
            args = self._delta_inputs(layer, h)
            if n_tok is None:
                o, layer["state"], _ = kda.prefill(*args, cu, S_in=layer["state"], dev_status=self.status)
            else:
                o = kda.decode(*(by_seq(t) for t in args), layer["state"], dev_status=self.status).to(torch.bfloat16)
        elif layer["kind"] == "decay":
            args, gate = self._decay_inputs(layer, h)
            seen = dict(norm_weight=layer["norm"], dev_status=self.status)
            if n_tok is None:
                o, _ = kda.lin_prefill(*args, cu, S_in=layer["state"], S_out=layer["state"], gate=gate, **seen)
            else:
                o = kda.lin_decode(*(by_seq(t) for t in args), layer["state"], n_commit=n_commit, gate=by_seq(gate),
                                   **seen).to(torch.bfloat16)
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
        return o

    def _step(self, x, cu, n_tok, n_commit=None):
        """x [T, width] bf16, packed by cu; n_tok: every sequence's tokens (decode), or None (prefill)."""
        new = cu.diff()
        kv_len = self.length + new
        if self.norms is not None:
            x = x.to(torch.float32, copy=True)  # the stack's own: the blocks' outputs are added in place
            h, x = kda.block_norm(x, self.norms[0]["pre"])
        for i, layer in enumerate(self.layers):
            if self.norms is None:
                h = torch.nn.functional.rms_norm(x.float(), (self.width,)).to(torch.bfloat16)
            y = self._mix(layer, h, cu, kv_len, n_tok, n_commit).reshape(-1, self.heads * D) @ layer["out"]
            if self.norms is None:
                x = x + y
            else:
                norm, after = self.norms[i], self.norms[i + 1]["pre"] if i + 1 < len(self.layers) else self.last_norm
                h, x = kda.block_norm(x, after, y, post_norm=True, post_weight=norm["post"], gate=h @ norm["gate"],
                                      scale=self.block_scale, x_out=x)
        self.length = kv_len if n_commit is None else self.length + n_commit
        return x if self.norms is None else h

    def prompt(self, x, cu_seqlens):
        """The next chunk of every sequence's prompt: x [T, width] bf16, cu_seqlens [n_seq + 1] int32."""
        return self._step(x, cu_seqlens, None)

    def decode(self, x, n_commit=None):
        """The next tokens: x [n_seq, n_tok, width] bf16, n_tok <= 4.  n_commit [n_seq] int32: how many of them each
        sequence keeps (None: all); a stack with delta layers keeps all."""
        if n_commit is not None and any(layer["kind"] == "delta" for layer in self.layers):
            raise ValueError("delta layers keep every token of a step: n_commit is for stacks without them")
        n, n_tok, _ = x.shape
        cu = torch.arange(0, n * n_tok + 1, n_tok, dtype=torch.int32, device=x.device)
        return self._step(x.reshape(-1, self.width), cu, n_tok, n_commit).view_as(x)


def serve(name, stack, prompts):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    print(f"{name}: {', '.join(layer['kind'] for layer in stack.layers)}")
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


def main():
    prompts = [300, 77, 1]
    serve("delta-rule stack", HybridStack(n_seq=len(prompts), max_tokens=1024), prompts)
    serve("decay stack", HybridStack(n_seq=len(prompts), max_tokens=1024, kinds=["decay", "decay", "attention", "decay"],
                                     post_norm=True, block_scale=0.5), prompts)


if __name__ == "__main__":
    main()
