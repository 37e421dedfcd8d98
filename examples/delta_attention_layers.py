"""Two layers of a hybrid stack served with this package's calls: the gated delta rule and softmax attention over a paged
cache, a prompt of packed sequences followed by single tokens.

    residual norm -> projection -> short convolution -> kda.gdn (gdn_step) -> gated norm -> projection
    residual norm -> projection -> qk_rope, kv_append -> attention (attn_step) -> projection

The delta rule's state and the cache are handed from the prompt to the steps and updated in place. A prompt's own attention
is plain torch here: it reads its keys and values back from the cache. Random weights; run it to see that steps after a
prompt give what one longer prompt gives:

    python examples/delta_attention_layers.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_linear_attention_kda_gb300 as kda  # noqa: E402

BF16 = torch.bfloat16


def param(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


class DeltaLayer:
    """q, k, v through the convolution, kda.gdn with two value heads to a key head, a norm per head and a SiLU gate."""

    def __init__(self, dim, heads, gen):
        self.H, self.HK = heads, heads // 2
        self.qkv, self.inner = (self.H + 2 * self.HK) * 128, self.H * 128
        self.norm = torch.ones(dim, device="cuda")
        self.w_in = param(gen, self.qkv + self.inner + 2 * self.H, dim, scale=dim ** -0.5, dtype=BF16)
        self.w_out = param(gen, dim, self.inner, scale=self.inner ** -0.5, dtype=BF16)
        self.taps = param(gen, self.qkv, 4, scale=0.5)
        self.A_log, self.dt_bias = torch.log(1 + 15 * torch.rand(self.H, generator=gen, device="cuda")), param(gen, self.H) - 4
        self.head_norm = torch.ones(128, device="cuda")

    def states(self, n, tokens):
        return {"conv": torch.zeros(n, 3, self.qkv, dtype=BF16, device="cuda"), "mixer": torch.zeros(n, self.H, 128, 128, device="cuda")}

    def __call__(self, h, st, positions, cu):
        row = torch.nn.functional.pad(h @ self.w_in.T, (0, -2 * self.H % 8))  # token rows keep 16-byte strides
        lead, step = row.shape[:-1], row.dim() == 2
        x = torch.empty(*lead, self.qkv, dtype=BF16, device=h.device)
        if step:
            kda.conv_step(row[..., :self.qkv], self.taps, x, st["conv"])
        else:
            kda.conv(row[..., :self.qkv], self.taps, x, initial_state=st["conv"], final_state=st["conv"], cu_seqlens=cu)
        n = self.HK * 128
        q, k, v = (t.unflatten(-1, (-1, 128)) for t in (x[..., :n], x[..., n:2 * n], x[..., 2 * n:]))
        z = row[..., self.qkv:self.qkv + self.inner].unflatten(-1, (self.H, 128))
        ab = row[..., self.qkv + self.inner:]
        a, beta = ab[..., :self.H], ab[..., self.H:2 * self.H]
        out = torch.empty(*lead, self.H, 128, dtype=BF16, device=h.device)
        args = (q, k, v, a, beta, 128 ** -0.5, out)
        if step:
            kda.gdn_step(*args, st["mixer"], self.A_log, self.dt_bias, qk_l2norm=True)
        else:
            kda.gdn(*args, self.A_log, self.dt_bias, st["mixer"], st["mixer"], cu, qk_l2norm=True)
        kda.gated_norm(out, z, self.head_norm, out, act="silu")
        return out.flatten(-2) @ self.w_out.T


class AttentionLayer:
    """Grouped queries with a norm per head, half of each head turned by its position, a cache of 16-token pages."""

    PAGE, D = 16, 64

    def __init__(self, dim, heads, gen):
        self.H, self.HK = heads, heads // 4
        self.norm = torch.ones(dim, device="cuda")
        self.w_in = param(gen, (self.H + 2 * self.HK) * self.D, dim, scale=dim ** -0.5, dtype=BF16)
        self.w_out = param(gen, dim, self.H * self.D, scale=(self.H * self.D) ** -0.5, dtype=BF16)
        self.q_norm, self.k_norm = (1 + param(gen, self.D, scale=0.1) for _ in range(2))
        self.inv_freq = (10000.0 ** (-torch.arange(0, 32, 2, dtype=torch.float64, device="cuda") / 32)).float()

    def states(self, n, tokens):
        pages = (tokens + self.PAGE - 1) // self.PAGE
        cache = torch.zeros(n * pages, 2, self.HK, self.PAGE, self.D, dtype=BF16, device="cuda")
        return {"k": cache[:, 0], "v": cache[:, 1], "table": torch.arange(n * pages, dtype=torch.int32, device="cuda").view(n, pages),
                "workspace": torch.empty(kda.attn_step_workspace_bytes(n, self.H, self.HK, self.D), dtype=torch.uint8, device="cuda")}

    def __call__(self, h, st, positions, cu):
        row = h @ self.w_in.T
        q, k, v = (t.unflatten(-1, (-1, self.D)) for t in row.split([self.H * self.D, self.HK * self.D, self.HK * self.D], -1))
        turned = torch.empty(q.shape, dtype=BF16, device=h.device)
        kda.qk_rope(q, None, turned, None, positions, self.inv_freq, self.q_norm)
        kda.kv_append(k, v, st["k"], st["v"], st["table"], positions, self.inv_freq, self.k_norm, norm=True, cu_seqlens=cu)
        out = torch.empty_like(turned)
        if h.dim() == 2:
            kda.attn_step(turned, st["k"], st["v"], st["table"], positions, out, self.D ** -0.5, workspace=st["workspace"])
        else:
            self.prompt_attention(turned, st, positions, cu, out)
        return out.flatten(-2) @ self.w_out.T

    def prompt_attention(self, q, st, positions, cu, out):
        for i, (b, e) in enumerate(zip(cu[:-1].tolist(), cu[1:].tolist())):
            pos = positions[0, b:e]
            k, v = (st[c][st["table"][i].long()].transpose(1, 2).flatten(0, 1).repeat_interleave(self.H // self.HK, 1).float() for c in ("k", "v"))
            x = torch.einsum("thd,shd->hts", q[0, b:e].float(), k) * self.D ** -0.5
            x = x.masked_fill(torch.arange(k.shape[0], device=x.device) > pos[None, :, None], -torch.inf)
            out[0, b:e] = torch.einsum("hts,shd->thd", torch.softmax(x, -1), v).to(BF16)


class Model:
    def __init__(self, dim=512, heads=8, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [DeltaLayer(dim, heads // 2, gen), AttentionLayer(dim, heads, gen)]
        self.last_norm = torch.ones(dim, device="cuda")

    def states(self, n, tokens):
        return [layer.states(n, tokens) for layer in self.layers]

    def __call__(self, embedded, states, positions, cu=None):
        """``embedded``: bf16 [1, T, dim] packed prompts with their ``cu``, or [S, dim] single tokens; ``positions`` alike.
        Returns the normed last rows; ``states`` are updated in place."""
        residual = embedded.float()
        h = torch.empty_like(embedded)
        kda.residual_norm(torch.zeros_like(embedded), residual, None, self.layers[0].norm, h)
        for i, layer in enumerate(self.layers):
            y = layer(h, states[i], positions, cu)
            norm = self.layers[i + 1].norm if i + 1 < len(self.layers) else self.last_norm
            kda.residual_norm(y, residual, residual, norm, h)
        return h


def packed(rows):
    """The prompts one behind the other, their bounds and the positions of their tokens."""
    cu = torch.tensor([0] + [len(r) for r in rows]).cumsum(0).cuda()
    return torch.cat(rows)[None], torch.cat([torch.arange(len(r)) for r in rows]).cuda()[None], cu


def main(steps=4):
    model = Model()
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = [torch.randn(n, 512, generator=gen, device="cuda").to(BF16) for n in (37, 300, 5, 161)]
    longest = max(len(r) for r in rows)
    # prompts of all but the last tokens of every row, then single tokens
    states = model.states(len(rows), longest)
    x, pos, cu = packed([r[:-steps] for r in rows])
    model(x, states, pos, cu)
    positions = torch.tensor([len(r) - steps for r in rows]).cuda()
    got = []
    for i in range(steps):
        got.append(model(torch.stack([r[len(r) - steps + i] for r in rows]), states, positions))
        positions += 1
    # the same tokens in one call
    x, pos, cu = packed(rows)
    whole = model(x, model.states(len(rows), longest), pos, cu)[0]
    want = torch.stack([o[-steps:] for o in whole.split([len(r) for r in rows])], 1)
    kda.check_device_status()
    rel = float((torch.stack(got).float() - want.float()).norm() / want.float().norm())
    print(f"4 prompts, {steps} steps each: steps against one longer prompt, relative difference {rel:.2e}")
    return rel


if __name__ == "__main__":
    main()
